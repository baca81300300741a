// qk_moe_few.cuh -- the experts' products for few assignments: two launches, no
// plan and no operands of the tensor cores, every product an fp32 multiply-add.
//
// A warp takes R rows of one assignment's expert (gate and up, or down); its
// lanes share out the row's units (Q4_K: 16 bytes, 32 values; Q8_0: half a block;
// Q6_K: 16 values), and the token's values of a unit stay in registers for all
// of the warp's rows.  A field of a word becomes a float by setting the exponent
// of 2^23 above it and taking 2^23 off again, which is exact; fields that lie
// higher in the word count 2^4, 2^8 or 2^12 times, and the token's value is
// scaled down by as much (exact, too, from magnitudes of 2^-114 on).
//
// The tokens' values lie in groups of 16, scaled so, with their sum behind them
// (Q4_K's minima meet sums of 32): five words of 16 bytes a group, so that lanes
// that read neighbouring groups meet no bank conflicts.  A thread block of the
// first launch makes them of its row of x, and 16 rows of h, one group, for the
// second.
//
// With so few assignments a call is bound by the time from one dependent load to
// the next and by its launches, so the second launch starts while the first runs
// and fetches its first weights before it waits for h.  One token of 8 of 128
// experts of 768 x 2048, Q4_K and Q6_K, calls one after another in a graph: 19.3
// us (24 MB of weights, 3.6 us at the memory's rate), where the plan and its
// launches take 38.2.  What bounds the first launch besides: each of its 384
// thread blocks lays out all of x for 32 rows, 37 KB of weights, and a lane has two
// units of a row to overlap.  Rows of a warp: 2 and 2 of gate and up, 4 of down (8
// of down: 1.2 us more a token).
#pragma once

#include "qk_moe.cuh"

namespace qk {
namespace moe {

constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewRows = 2;                        // gate rows (and as many up rows) of a warp
constexpr int kFewDownRows = 4;

// Loads of weights: not moved over the wait for the launch before.
__device__ __forceinline__ uint4 ldw128(const uint8_t *p)
{
    uint4 v;
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ldw16(const uint8_t *p)
{
    uint16_t v;
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ int ldw8(const uint8_t *p)
{
    int v;
    asm volatile("ld.global.nc.s8 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

struct Pair {
    uint64_t v;
};
__device__ __forceinline__ Pair pair_of(float a, float b)
{
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(a), "f"(b));
    return p;
}
__device__ __forceinline__ float sum_of(Pair p)
{
    float a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v));
    return a + b;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b)
{
    Pair p;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p.v) : "l"(a.v), "l"(b.v));
    return p;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c)
{
    Pair p;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return p;
}
// The field of w under MASK (below bit 23) above 2^23
template <uint32_t MASK>
__device__ __forceinline__ float field(uint32_t w)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(MASK), "n"(0x4B000000));
    return __uint_as_float(r);
}
constexpr float kFieldOff = -8388608.0f;
template <uint32_t A, uint32_t B>
__device__ __forceinline__ Pair fields(uint32_t w)
{
    return add2(pair_of(field<A>(w), field<B>(w)), pair_of(kFieldOff, kFieldOff));
}
// bytes I and I + 1 of w less `bias`
template <int I>
__device__ __forceinline__ Pair bytes_less(uint32_t w, float bias)
{
    return add2(pair_of(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540 + I)), __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7541 + I))),
                pair_of(kFieldOff - bias, kFieldOff - bias));
}

constexpr int kGroup = 16, kGroupPitch = 20;       // values, and floats they take
constexpr int kFewBlock = 256;                     // a row of groups is whole runs of this many values
__host__ __device__ constexpr int64_t few_pitch(int64_t cols) { return (cols + kFewBlock - 1) / kFewBlock * (kFewBlock / kGroup) * kGroupPitch; }
// what value k of a row is scaled by
template <int FMT>
__device__ __forceinline__ float few_factor(int k)
{
    return FMT == kFmtQ4K ? (k & 32 ? 0x1p-4f : 1.0f) * (k & 1 ? 0x1p-8f : 1.0f) : 1.0f;
}

template <int FMT>
struct FewUnit;

template <>
struct FewUnit<kFmtQ4K> {
    static constexpr int kPerBlock = 8, kBlock = 256;
    struct Raw {
        uint4 head, q;
    };
    struct X {
        float4 lo[4], hi[4];
        float sum_lo, sum_hi;
    };
    static __device__ __forceinline__ void load(Raw &r, const uint8_t *row, int u)
    {
        const uint8_t *p = row + (u >> 3) * 144;
        r.head = ldw128(p), r.q = ldw128(p + 16 + 16 * (u & 7));
    }
    static __device__ __forceinline__ void load(X &x, const float *row, int u)
    {
        const float *p = row + ((u >> 1) * 4 + (u & 1)) * kGroupPitch;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x.lo[i] = *reinterpret_cast<const float4 *>(p + 4 * i);
            x.hi[i] = *reinterpret_cast<const float4 *>(p + 2 * kGroupPitch + 4 * i);
        }
        x.sum_lo = p[kGroup], x.sum_hi = p[2 * kGroupPitch + kGroup];
    }
    static __device__ __forceinline__ float dot(const Raw &r, const X &x, int u)
    {
        Pair lo = {0}, hi = {0};
        const uint32_t w[4] = {r.q.x, r.q.y, r.q.z, r.q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v = w[i] >> 16;
            lo = fma2(fields<0x000f, 0x0f00>(w[i]), pair_of(x.lo[i].x, x.lo[i].y), lo);
            hi = fma2(fields<0x00f0, 0xf000>(w[i]), pair_of(x.hi[i].x, x.hi[i].y), hi);
            lo = fma2(fields<0x000f, 0x0f00>(v), pair_of(x.lo[i].z, x.lo[i].w), lo);
            hi = fma2(fields<0x00f0, 0xf000>(v), pair_of(x.hi[i].z, x.hi[i].w), hi);
        }
        // sub-blocks 2j and 2j + 1 of the super-block: six bits each of scale and minimum
        const int j = (u & 7) >> 1, sh = (j & 1) * 16;
        const uint32_t A = r.head.y >> sh, B = r.head.z >> sh, C = r.head.w >> sh;
        const uint32_t sc = j < 2 ? A & 0x3f3fu : (C & 0x0f0fu) | ((A >> 2) & 0x3030u);
        const uint32_t m = j < 2 ? B & 0x3f3fu : ((C >> 4) & 0x0f0fu) | ((B >> 2) & 0x3030u);
        const float2 d = __half22float2(*reinterpret_cast<const __half2 *>(&r.head.x));
        const float s0 = field<0x00ff>(sc) + kFieldOff, s1 = field<0x00ff>(sc >> 8) + kFieldOff;
        const float m0 = field<0x00ff>(m) + kFieldOff, m1 = field<0x00ff>(m >> 8) + kFieldOff;
        return d.x * fmaf(s0, sum_of(lo), s1 * sum_of(hi)) - d.y * fmaf(m0, x.sum_lo, m1 * x.sum_hi);
    }
};

template <>
struct FewUnit<kFmtQ80> {
    static constexpr int kPerBlock = 2, kBlock = 32;
    struct Raw {
        uint32_t q[4], d;
    };
    struct X {
        float4 v[4];
    };
    static __device__ __forceinline__ void load(Raw &r, const uint8_t *row, int u)
    {
        const uint8_t *p = row + static_cast<int64_t>(u >> 1) * 34;
        r.d = ldw16(p);
        p += 2 + 16 * (u & 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.q[i] = ldw16(p + 4 * i) | ldw16(p + 4 * i + 2) << 16;
    }
    static __device__ __forceinline__ void load(X &x, const float *row, int u)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) x.v[i] = *reinterpret_cast<const float4 *>(row + u * kGroupPitch + 4 * i);
    }
    static __device__ __forceinline__ float dot(const Raw &r, const X &x, int)
    {
        Pair a = {0}, b = {0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = r.q[i] ^ 0x80808080u;
            a = fma2(bytes_less<0>(w, 128.0f), pair_of(x.v[i].x, x.v[i].y), a);
            b = fma2(bytes_less<2>(w, 128.0f), pair_of(x.v[i].z, x.v[i].w), b);
        }
        return half_bits_to_float(static_cast<uint16_t>(r.d)) * sum_of(add2(a, b));
    }
};

template <>
struct FewUnit<kFmtQ6K> {
    static constexpr int kPerBlock = 16, kBlock = 256;
    struct Raw {
        uint32_t a, b, h, d;
        int s[4];
    };
    struct X {
        float4 v[4];
    };
    static __device__ __forceinline__ void load(Raw &r, const uint8_t *row, int u)
    {
        const uint8_t *p = row + static_cast<int64_t>(u >> 4) * 210;
        const int n = (u >> 3) & 1, l = u & 7;
        const auto word = [](const uint8_t *q) { return ldw16(q) | ldw16(q + 2) << 16; };
        r.a = word(p + 64 * n + 4 * l), r.b = word(p + 64 * n + 32 + 4 * l), r.h = word(p + 128 + 32 * n + 4 * l);
#pragma unroll
        for (int t = 0; t < 4; ++t) r.s[t] = ldw8(p + 192 + 8 * n + 2 * t + (l >> 2));
        r.d = ldw16(p + 208);
    }
    static __device__ __forceinline__ void load(X &x, const float *row, int u)
    {
        const int k = (u >> 4) * 256 + 128 * ((u >> 3) & 1) + 4 * (u & 7);
#pragma unroll
        for (int t = 0; t < 4; ++t) x.v[t] = *reinterpret_cast<const float4 *>(row + ((k >> 4) + 2 * t) * kGroupPitch + (k & 15));
    }
    static __device__ __forceinline__ float dot(const Raw &r, const X &x, int)
    {
        float sum = 0.0f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint32_t low = ((t & 1 ? r.b : r.a) >> (t & 2 ? 4 : 0)) & 0x0f0f0f0fu;
            const uint32_t w = low | ((t < 2 ? r.h << (4 - 2 * t) : r.h >> (2 * t - 4)) & 0x30303030u);
            const Pair a = fma2(bytes_less<0>(w, 32.0f), pair_of(x.v[t].x, x.v[t].y), Pair{0});
            const float scale = __uint_as_float(0x4B000000u + (r.s[t] + 128)) - (8388608.0f + 128.0f);
            sum = fmaf(scale, sum_of(fma2(bytes_less<2>(w, 32.0f), pair_of(x.v[t].z, x.v[t].w), a)), sum);
        }
        return half_bits_to_float(static_cast<uint16_t>(r.d)) * sum;
    }
};

// Units u, u + step, ... of R rows: the sums of this lane.  The first units' weights are fetched before `ready` is called,
// and with AHEAD the next ones' before a unit's products.
template <int FMT, bool AHEAD, int R, class Ready>
__device__ __forceinline__ void few_products(float (&sum)[R], const uint8_t *const (&rows)[R], int u, int step, int units,
                                             const float *x, Ready ready)
{
    using Unit = FewUnit<FMT>;
    typename Unit::Raw raw[R];
    const auto fetch = [&](typename Unit::Raw (&to)[R], int n) {
        if (n < units) {
#pragma unroll
            for (int r = 0; r < R; ++r) Unit::load(to[r], rows[r], n);
        }
    };
#pragma unroll
    for (int r = 0; r < R; ++r) sum[r] = 0.0f;
    fetch(raw, u);
    ready();
    while (u < units) {
        typename Unit::X v;
        Unit::load(v, x, u);
        if constexpr (AHEAD) {
            typename Unit::Raw next[R];
            fetch(next, u + step);
#pragma unroll
            for (int r = 0; r < R; ++r) sum[r] += Unit::dot(raw[r], v, u), raw[r] = next[r];
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) sum[r] += Unit::dot(raw[r], v, u);
            fetch(raw, u + step);
        }
        u += step;
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int d = 16; d > 0; d /= 2) sum[r] += __shfl_xor_sync(~0u, sum[r], d);
}

// h[a] = silu(gate x) * (up x), in groups as the down products (of format DOWN) want them: block (b, a), 16 rows.
template <int FMT, int DOWN>
__global__ void __launch_bounds__(kFewThreads) few_gate_kernel(const FewArgs a)
{
    static_assert(kFewWarps * kFewRows == kGroup, "a thread block makes a group of h");
    extern __shared__ __align__(16) float row_x[];
    __shared__ float group[kGroup];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    wait_for_previous();
    let_next_start();                          // what came before this launch is done: the next may read the ids at once
    const int64_t p = blockIdx.y;
    const int id = a.ids[p];
    if (id >= a.experts && blockIdx.x == 0 && threadIdx.x == 0) record_error(a.err, kErrBadIndex);
    if (id < 0 || id >= a.experts) return;
    const int row0 = blockIdx.x * kGroup + warp * kFewRows;
    if (static_cast<int>(blockIdx.x) * kGroup < a.rows) {
        const uint8_t *rows[2 * kFewRows];
#pragma unroll
        for (int r = 0; r < kFewRows; ++r) {
            const int64_t row = min(row0 + r, a.rows - 1);
            rows[r] = a.a.w + (id * a.a.expert_rows + row) * a.a.row_bytes;
            rows[kFewRows + r] = a.b.w + (id * a.b.expert_rows + row) * a.b.row_bytes;
        }
        using Unit = FewUnit<FMT>;
        float sum[2 * kFewRows];
        few_products<FMT, true>(sum, rows, lane, 32, (a.cols + Unit::kBlock - 1) / Unit::kBlock * Unit::kPerBlock, row_x, [&] {
            const int64_t at = p / a.top_k * a.ldx;
            for (int k = threadIdx.x * 4; k < (a.cols + kFewBlock - 1) / kFewBlock * kFewBlock; k += kFewThreads * 4) {
                float4 v = four(a.x, at, k, a.cols, a.x_type, a.vec);
                float s = (v.x + v.y) + (v.z + v.w);
                s += __shfl_xor_sync(~0u, s, 1), s += __shfl_xor_sync(~0u, s, 2);
                v.x *= few_factor<FMT>(k), v.y *= few_factor<FMT>(k + 1), v.z *= few_factor<FMT>(k + 2), v.w *= few_factor<FMT>(k + 3);
                float *to = row_x + (k >> 4) * kGroupPitch;
                *reinterpret_cast<float4 *>(to + (k & 15)) = v;
                if (FMT == kFmtQ4K && (k & 15) == 0) to[kGroup] = s;
            }
            __syncthreads();
        });
        if (lane == 0)
#pragma unroll
            for (int r = 0; r < kFewRows; ++r) group[warp * kFewRows + r] = row0 + r < a.rows ? silu(sum[r]) * sum[kFewRows + r] : 0.0f;
    } else if (lane < kFewRows) {
        group[warp * kFewRows + lane] = 0.0f;  // past the last row
    }
    __syncthreads();
    float *out = a.h + p * few_pitch(a.rows) + blockIdx.x * kGroupPitch;
    if (threadIdx.x < kGroup) out[threadIdx.x] = group[threadIdx.x] * few_factor<DOWN>(blockIdx.x * kGroup + threadIdx.x);
    if (threadIdx.x == kGroup) {
        float s = 0.0f;
        for (int i = 0; i < kGroup; i += 4) s += (group[i] + group[i + 1]) + (group[i + 2] + group[i + 3]);
        out[kGroup] = s;
    }
}

// y[t] = sum over j, in order, of weights[t][j] * (down h of (t, j)): block (b, t), a warp one j (or a part of its units).
template <int FMT>
__global__ void __launch_bounds__(kFewThreads) few_down_kernel(const FewArgs a)
{
    constexpr int R = kFewDownRows;
    __shared__ float parts[(kMaxFew + kFewWarps) * R];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = blockIdx.y;
    const int row0 = blockIdx.x * R;
    const int split = max(1, kFewWarps / a.top_k), items = a.top_k * split;
    using Unit = FewUnit<FMT>;
    const int units = (a.cols + Unit::kBlock - 1) / Unit::kBlock * Unit::kPerBlock;
    bool waited = false;
    let_next_start();
    for (int i = warp; i < items; i += kFewWarps) {
        const int64_t p = t * a.top_k + i / split;
        const int id = a.ids[p];
        if (id < 0 || id >= a.experts) continue;
        const uint8_t *rows[R];
#pragma unroll
        for (int r = 0; r < R; ++r)
            rows[r] = a.a.w + (id * a.a.expert_rows + min(row0 + r, a.rows - 1)) * a.a.row_bytes;
        float sum[R];
        few_products<FMT, false>(sum, rows, lane + 32 * (i % split), 32 * split, units,
                          a.h + p * few_pitch(a.cols), [&] {
                              if (!waited) wait_for_previous();
                              waited = true;
                          });
        if (lane < R) {
            float v = sum[0];
#pragma unroll
            for (int r = 1; r < R; ++r) v = lane == r ? sum[r] : v;
            parts[i * R + lane] = v;
        }
    }
    if (!waited) wait_for_previous();
    __syncthreads();
    if (threadIdx.x < R && row0 + static_cast<int>(threadIdx.x) < a.rows) {
        float y = 0.0f;
        for (int j = 0; j < a.top_k; ++j) {
            const int id = a.ids[t * a.top_k + j];
            if (id < 0) continue;
            float v = id < a.experts ? 0.0f : __int_as_float(0x7fc00000);
            for (int s = 0; s < split && id < a.experts; ++s) v += parts[(j * split + s) * R + threadIdx.x];
            y += a.weights[t * a.top_k + j] * v;
        }
        store_float_as(a.y, t * a.ldy + row0 + threadIdx.x, a.y_type, y);
    }
}

template <int FMT>
cudaError_t few_gate(const FewArgs &a, int64_t A, int down, bool chained, cudaStream_t st)
{
    const dim3 grid((a.rows + kFewBlock - 1) / kFewBlock * (kFewBlock / kGroup), static_cast<unsigned>(A));
    const size_t smem = sizeof(float) * few_pitch(a.cols);
    const auto kern = down == kFmtQ4K ? few_gate_kernel<FMT, kFmtQ4K> : few_gate_kernel<FMT, kFmtQ80>;     // (Q6_K as Q8_0)
    return launch_chained(kern, grid, kFewThreads, smem, st, chained, a);
}
template <int FMT>
cudaError_t few_down(const FewArgs &a, int64_t T, cudaStream_t st)
{
    return launch_chained(few_down_kernel<FMT>, dim3((a.rows + kFewDownRows - 1) / kFewDownRows, static_cast<unsigned>(T)), kFewThreads, 0,
                          st, true, a);
}

}  // namespace moe
}  // namespace qk
