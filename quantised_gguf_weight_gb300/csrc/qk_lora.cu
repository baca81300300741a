// qk_lora.cu -- low-rank adapters of many requests beside a shared projection:
//   out[t] = y[t] + scale[a] * B[a] (A[a] x[t]),  a = ids[t].
//
// Two forms.  In one launch a cluster of thread blocks takes a tile of
// neighbouring tokens and one adapter after another of those that the tile has:
// each block forms its columns' part of V = A x (rank values a token), the blocks
// add the parts through distributed shared memory, always in their order, and
// each adds its columns of B V to y.  In two launches V lies in memory between
// them (below); two_launches() says which calls take which.
//
// Few tokens are bound by latency: one token beside 4096 x 6144, rank 16, 8.2 us
// (6.3 in a graph; 12.3 before clusters shared its columns), 64 of 48 adapters
// 22.6 (8 MB of adapters, 2.3 us at the memory's rate; of the 512 blocks 304 are
// resident at once.  Clusters of 4, which all would be, took 20.5 for 22.5, but
// 255 tokens of 4 adapters 58 us for 24).
//
// The products are m16n8k8 in tf32, which holds 16-bit adapters and activations
// exactly; fp32 operands, and V, are two tf32 pieces (22 bits).  A lane's values
// of an operand are neighbours in memory: which columns a product's slots stand
// for is free as long as both operands agree.
#include <algorithm>
#include <cmath>

#include "qk_kv4.cuh"
#include "qk_moe.cuh"
#include "qk_tc.cuh"

namespace qk {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kCluster = 8;
constexpr int kBlockRank = 64;                 // ranks of a pass of the first product
constexpr int kMaxRank = 256;

struct LoraArgs {
    const void *x, *y, *A, *B;
    void *out;
    int64_t ldx, ldy, ldo, T, n_adapters;
    int x_type, y_type, w_type, K, N, rank;
    const int32_t *ids;
    const float *scales;
    int steps, cuts;                           // clusters that share a tile's adapters, and their columns of y
    float *V;                                  // many tokens: [T][ranks, padded] of scale A x
    bool vec_x, vec_y, vec_a, vec_b;
    int *err;
};

__device__ __forceinline__ uint32_t tf32_of(float v)
{
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ void mma8(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Q neighbouring values of a row from element i on, 0 from element `n` (of the row) on.  WIDE: fp32.
template <int Q, bool WIDE>
__device__ __forceinline__ void load_values(float (&v)[Q], const void *base, int64_t row, int i, int n, bool vec, bool half)
{
    if (vec && i + Q <= n) {
        if constexpr (WIDE) {
            const float *p = static_cast<const float *>(base) + row + i;
#pragma unroll
            for (int k = 0; k < Q; k += 4)
                if constexpr (Q >= 4) {
                    const float4 f = __ldg(reinterpret_cast<const float4 *>(p + k));
                    v[k] = f.x, v[k + 1] = f.y, v[k + 2] = f.z, v[k + 3] = f.w;
                } else {
                    const float2 f = __ldg(reinterpret_cast<const float2 *>(p + k));
                    v[k] = f.x, v[k + 1] = f.y;
                }
        } else {
            const uint16_t *p = static_cast<const uint16_t *>(base) + row + i;
            uint32_t w[Q / 2];
            if constexpr (Q >= 8) {
#pragma unroll
                for (int k = 0; k < Q / 8; ++k) {
                    const uint4 f = __ldg(reinterpret_cast<const uint4 *>(p) + k);
                    w[4 * k] = f.x, w[4 * k + 1] = f.y, w[4 * k + 2] = f.z, w[4 * k + 3] = f.w;
                }
            } else if constexpr (Q == 4) {
                const uint2 f = __ldg(reinterpret_cast<const uint2 *>(p));
                w[0] = f.x, w[1] = f.y;
            } else {
                w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
            }
#pragma unroll
            for (int k = 0; k < Q / 2; ++k) {
                const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
                v[2 * k] = half ? h.x : __uint_as_float(w[k] << 16);
                v[2 * k + 1] = half ? h.y : __uint_as_float(w[k] & 0xffff0000u);
            }
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < Q; ++k)
        v[k] = i + k < n ? load_as_float(base, row + i + k, WIDE ? QK_F32 : half ? QK_F16 : QK_BF16) : 0.0f;
}

// d += a b, of fp32 values in one or two tf32 pieces (PA, PB of them count).
template <int PA, int PB>
__device__ __forceinline__ void mma_pieces(float (&d)[4], const float (&a)[4], float b0, float b1)
{
    uint32_t ah[4], al[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        ah[i] = PA == 2 ? tf32_of(a[i]) : __float_as_uint(a[i]);
        if constexpr (PA == 2) al[i] = tf32_of(a[i] - __uint_as_float(ah[i]));
    }
    const uint32_t h0 = PB == 2 ? tf32_of(b0) : __float_as_uint(b0), h1 = PB == 2 ? tf32_of(b1) : __float_as_uint(b1);
    mma8(d, ah, h0, h1);
    if constexpr (PA == 2) mma8(d, al, h0, h1);
    if constexpr (PB == 2) mma8(d, ah, tf32_of(b0 - __uint_as_float(h0)), tf32_of(b1 - __uint_as_float(h1)));
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool half)
{
    if (half) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack16(uint32_t w, bool half)
{
    if (half) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ float4 read_remote(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

// MT: 16-row tiles of tokens; NR: 8-rank tiles of a pass; XW, WW: activations and adapters in fp32.
template <int MT, int NR, bool XW, bool WW>
__global__ void __launch_bounds__(kThreads) lora_kernel(const LoraArgs a)
{
    constexpr int ROWS = 16 * MT, R8 = 8 * NR;
    extern __shared__ __align__(16) float smem[];
    __shared__ int ids[ROWS], list[ROWS], n_list;
    const int blocks = (a.rank + R8 - 1) / R8, width = blocks * R8, pitch = width + 4;
    float *parts = smem;                                     // [warp][ROWS][R8]
    float *mine = parts + kWarps * ROWS * R8;                // [ROWS][width]: this block's part of V
    float *V = mine + ROWS * width;                          // [ROWS][pitch]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int rank = static_cast<int>(cluster_ctarank());
    const int64_t cluster = blockIdx.x / kCluster;
    const int cut = static_cast<int>(cluster % a.cuts), step = static_cast<int>(cluster / a.cuts % a.steps);
    const int64_t t0 = cluster / a.cuts / a.steps * ROWS;
    moe::let_next_start();
    moe::wait_for_previous();
    if (tid == 0) n_list = 0;
    if (tid < ROWS) ids[tid] = t0 + tid < a.T ? a.ids[t0 + tid] : -1;
    __syncthreads();
    if (tid < 32)
        for (int base = 0; base < ROWS; base += 32) {        // the tile's adapters, in the order of their first tokens
            const int i = base + lane;
            const int id = i < ROWS ? ids[i] : -1;
            bool first = id >= 0 && id < a.n_adapters;
            for (int k = 0; k < i && first; ++k) first = ids[k] != id;
            const unsigned who = __ballot_sync(~0u, first);
            if (first) list[n_list + __popc(who & ((1u << lane) - 1))] = id;
            __syncwarp();
            if (lane == 0) n_list += __popc(who);
            __syncwarp();
        }
    __syncthreads();
    const int n_adapters = n_list;
    // columns of this block: of x, and of y
    const int k_per = ((a.K + kCluster - 1) / kCluster + 31) / 32 * 32, k0 = min(a.K, rank * k_per), k1 = min(a.K, k0 + k_per);
    const int parts_n = kCluster * a.cuts, n_per = ((a.N + parts_n - 1) / parts_n + 15) / 16 * 16;
    const int n0 = min(a.N, (cut * kCluster + rank) * n_per), n1 = min(a.N, n0 + n_per);
    const bool x_half = a.x_type == QK_F16, w_half = a.w_type == QK_F16;

    if (step == 0) {
        // rows without an adapter
        for (int base = 0; base < ROWS; base += 32) {
            const int r = base + lane;
            unsigned none = __ballot_sync(~0u, r < ROWS && t0 + r < a.T && (ids[r < ROWS ? r : 0] < 0 || ids[r < ROWS ? r : 0] >= a.n_adapters));
            for (; none; none &= none - 1) {
                const int i = base + __ffs(none) - 1;
                const int64_t t = t0 + i;
                const bool bad = ids[i] >= 0;
                if (bad && tid == 0 && rank == 0) record_error(a.err, kErrBadIndex);
                if (bad || a.out != a.y)
                    for (int n = n0 + tid; n < n1; n += kThreads)
                        store_float_as(a.out, t * a.ldo + n, a.y_type,
                                       bad ? __int_as_float(0x7fc00000) : load_as_float(a.y, t * a.ldy + n, a.y_type));
            }
        }
    }

    for (int j = step; j < n_adapters; j += a.steps) {
        const int id = list[j];
        const int64_t a_row = static_cast<int64_t>(id) * a.rank, b_row = static_cast<int64_t>(id) * a.N;
        for (int rb = 0; rb < blocks; ++rb) {
            float acc[MT][NR][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
            struct Turn {
                float x[MT][2][8], w[NR][8];
            };
            const auto load = [&](Turn &t, int k) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int row = m * 16 + h * 8 + g;
                        if (ids[row] == id) load_values<8, XW>(t.x[m][h], a.x, (t0 + row) * a.ldx, k + 8 * c, a.K, a.vec_x, x_half);
                        else {
#pragma unroll
                            for (int i = 0; i < 8; ++i) t.x[m][h][i] = 0.0f;
                        }
                    }
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    const int r = rb * R8 + n * 8 + g;
                    if (r < a.rank) load_values<8, WW>(t.w[n], a.A, (a_row + r) * a.K, k + 8 * c, a.K, a.vec_a, w_half);
                    else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) t.w[n][i] = 0.0f;
                    }
                }
            };
            const auto products = [&](const Turn &t) {
#pragma unroll
                for (int s = 0; s < 4; ++s)
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const float xa[4] = {t.x[m][0][2 * s], t.x[m][1][2 * s], t.x[m][0][2 * s + 1], t.x[m][1][2 * s + 1]};
                            mma_pieces<XW ? 2 : 1, WW ? 2 : 1>(acc[m][n], xa, t.w[n][2 * s], t.w[n][2 * s + 1]);
                        }
            };
            // a turn ahead where registers allow
            if constexpr (MT * 2 + NR <= 6) {
                int k = k0 + warp * 32;
                Turn next;
                if (k < k1) load(next, k);
                for (; k < k1; k += kWarps * 32) {
                    const Turn t = next;
                    if (k + kWarps * 32 < k1) load(next, k + kWarps * 32);
                    products(t);
                }
            } else {
                for (int k = k0 + warp * 32; k < k1; k += kWarps * 32) {
                    Turn t;
                    load(t, k);
                    products(t);
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        *reinterpret_cast<float2 *>(parts + (warp * ROWS + m * 16 + h * 8 + g) * R8 + n * 8 + 2 * c) =
                            make_float2(acc[m][n][2 * h], acc[m][n][2 * h + 1]);
            __syncthreads();
            for (int i = tid; i < ROWS * R8; i += kThreads) {
                float s = parts[i];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) s += parts[w * ROWS * R8 + i];
                mine[i / R8 * width + rb * R8 + i % R8] = s;
            }
            __syncthreads();
        }
        cluster_sync();
        const float scale = a.scales ? a.scales[id] : 1.0f;
        const uint32_t at = smem_u32(mine);
        for (int i = tid * 4; i < ROWS * width; i += kThreads * 4) {
            float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float4 p[kCluster];
#pragma unroll
            for (int q = 0; q < kCluster; ++q) p[q] = read_remote(mapa_shared(at + 4 * i, q));
#pragma unroll
            for (int q = 0; q < kCluster; ++q) s.x += p[q].x, s.y += p[q].y, s.z += p[q].z, s.w += p[q].w;
            *reinterpret_cast<float4 *>(V + i / width * pitch + i % width) =
                make_float4(s.x * scale, s.y * scale, s.z * scale, s.w * scale);
        }
        cluster_sync();                                      // everyone has read: the parts may be written again
        // 16 columns a turn: lane c of a row gets four neighbours
        for (int n = n0 + warp * 16; n < n1; n += kWarps * 16) {
            float acc[MT][2][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[m][q][i] = 0.0f;
            for (int rb = 0; rb < blocks; ++rb) {
                float bv[2][2 * NR];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int col = n + 4 * (g >> 1) + 2 * q + (g & 1);
                    if (col < a.N)
                        load_values<2 * NR, WW>(bv[q], a.B, (b_row + col) * a.rank, rb * R8 + 2 * NR * c, a.rank, a.vec_b, w_half);
                    else {
#pragma unroll
                        for (int i = 0; i < 2 * NR; ++i) bv[q][i] = 0.0f;
                    }
                }
#pragma unroll
                for (int s = 0; s < NR; ++s)
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const float2 u = *reinterpret_cast<const float2 *>(V + (m * 16 + g) * pitch + rb * R8 + 2 * NR * c + 2 * s);
                        const float2 w = *reinterpret_cast<const float2 *>(V + (m * 16 + 8 + g) * pitch + rb * R8 + 2 * NR * c + 2 * s);
                        const float va[4] = {u.x, w.x, u.y, w.y};
#pragma unroll
                        for (int q = 0; q < 2; ++q) mma_pieces<2, WW ? 2 : 1>(acc[m][q], va, bv[q][2 * s], bv[q][2 * s + 1]);
                    }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = m * 16 + h * 8 + g;
                    if (ids[row] != id) continue;
                    const int64_t from = (t0 + row) * a.ldy, to = (t0 + row) * a.ldo;
                    const int col = n + 4 * c;
                    const float d[4] = {acc[m][0][2 * h], acc[m][0][2 * h + 1], acc[m][1][2 * h], acc[m][1][2 * h + 1]};
                    if (a.vec_y && col + 4 <= a.N) {
                        if (a.y_type == QK_F32) {
                            float4 f = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.y) + from + col);
                            f.x += d[0], f.y += d[1], f.z += d[2], f.w += d[3];
                            *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + to + col) = f;
                        } else {
                            const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.y) + from + col);
                            uint2 o;
                            if (a.y_type == QK_F16) {
                                const float2 f0 = __half22float2(*reinterpret_cast<const __half2 *>(&w.x));
                                const float2 f1 = __half22float2(*reinterpret_cast<const __half2 *>(&w.y));
                                const __half2 r0 = __floats2half2_rn(f0.x + d[0], f0.y + d[1]), r1 = __floats2half2_rn(f1.x + d[2], f1.y + d[3]);
                                o = make_uint2(*reinterpret_cast<const uint32_t *>(&r0), *reinterpret_cast<const uint32_t *>(&r1));
                            } else {
                                const __nv_bfloat162 r0 = __floats2bfloat162_rn(__uint_as_float(w.x << 16) + d[0], __uint_as_float(w.x & 0xffff0000u) + d[1]);
                                const __nv_bfloat162 r1 = __floats2bfloat162_rn(__uint_as_float(w.y << 16) + d[2], __uint_as_float(w.y & 0xffff0000u) + d[3]);
                                o = make_uint2(*reinterpret_cast<const uint32_t *>(&r0), *reinterpret_cast<const uint32_t *>(&r1));
                            }
                            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + to + col) = o;
                        }
                    } else {
                        for (int i = 0; i < 4 && col + i < a.N; ++i)
                            store_float_as(a.out, to + col + i, a.y_type, load_as_float(a.y, from + col + i, a.y_type) + d[i]);
                    }
                }
        }
        __syncthreads();                                     // V is read to the end
    }
}

template <int MT, int NR, bool XW, bool WW>
cudaError_t launch_as(const LoraArgs &a, cudaStream_t st)
{
    constexpr int ROWS = 16 * MT, R8 = 8 * NR;
    const int width = (a.rank + R8 - 1) / R8 * R8;
    const size_t smem = sizeof(float) * (kWarps * ROWS * R8 + ROWS * width + ROWS * (width + 4));
    const auto kern = lora_kernel<MT, NR, XW, WW>;
    static SharedGrant granted;                              // (the size goes with the rank)
    cudaError_t e = granted.at_least(kern, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    const int64_t tiles = (a.T + ROWS - 1) / ROWS;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * a.steps * a.cuts * kCluster)), cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem, cfg.stream = st;
    cudaLaunchAttribute at[2]{};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kCluster, at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at, cfg.numAttrs = library_programmatic() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

// ---------------------------------------------------------------- many tokens
// Two launches with V = scale A x in memory between them.  The first: a thread
// block has a tile of tokens, its warps every eighth 32 columns of x and A; the
// warps' sums are added in their order.  The second: V's rows stay in a warp's
// registers as the products' operand while it goes over its columns of B and y.
// A tile's adapters are shared out over blocks, each for its own rows.
//
// Where x and the adapters have one 16-bit type the products are m16n8k16 in it,
// operands as they lie in memory; else the first launch's are tf32, as above.
// In the second 16-bit adapters meet V as two fp16 pieces below its row's
// largest, or three bf16 ones, fp32 ones as two of tf32: 22 bits or more.  Beside
// bf16 outputs bf16 adapters meet two, 2^-17 of V, eight bits below the outputs'
// own rounding (with three, 4096 tokens of rank 64 take 61 us in a graph for 55).
//
// The kernels here load straight into the products' registers and take any
// alignment; the ones with rings further down do the same products in the same
// order.  4096 bf16 tokens of 7 requests beside 4096 x 6144, rank 64: 24 and 36
// us, 57 together, for 140 MB (21 us at the memory's rate; the tensor cores are
// 16% and 31% busy).  Every 32 tokens read A and B again, 167 MB more from L2, and
// the first launch is one round of 128 working blocks, whose start and whose sum
// over eight warps overlap with nothing.

constexpr int kTallRows = 32, kShrinkRows = 16;            // tokens of a block of the second, and of the first launch

struct TileList {
    int ids[kTallRows], list[kTallRows], n;
};
// The tile's ids, and its adapters in the order of their first tokens.
__device__ __forceinline__ void list_adapters(TileList &l, const LoraArgs &a, int64_t t0, int rows)
{
    const int tid = threadIdx.x;
    if (tid < kTallRows) {
        const int id = tid < rows && t0 + tid < a.T ? a.ids[t0 + tid] : -1;
        l.ids[tid] = id;
        __syncwarp();
        const unsigned same = __match_any_sync(~0u, id);
        const bool first = id >= 0 && id < a.n_adapters && tid == __ffs(same) - 1;
        const unsigned who = __ballot_sync(~0u, first);
        if (first) l.list[__popc(who & ((1u << tid) - 1))] = id;
        if (tid == 0) l.n = __popc(who);
    }
    __syncthreads();
}

constexpr int kBf16 = 0, kF16 = 1, kTf32 = 2;      // products' type

template <int TYPE>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    if constexpr (TYPE == kF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Q neighbouring 16-bit values of a row as they are, 0 from element n on.
template <int Q>
__device__ __forceinline__ void load_raw(uint32_t (&w)[Q / 2], const void *base, int64_t row, int i, int n, bool vec)
{
    const uint16_t *p = static_cast<const uint16_t *>(base) + row + i;
    if (vec && i + Q <= n) {
        if constexpr (Q >= 8) {
#pragma unroll
            for (int k = 0; k < Q / 8; ++k) {
                const uint4 f = __ldg(reinterpret_cast<const uint4 *>(p) + k);
                w[4 * k] = f.x, w[4 * k + 1] = f.y, w[4 * k + 2] = f.z, w[4 * k + 3] = f.w;
            }
        } else {
            const uint2 f = __ldg(reinterpret_cast<const uint2 *>(p));
            w[0] = f.x, w[1] = f.y;
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < Q / 2; ++k)
        w[k] = (i + 2 * k < n ? __ldg(p + 2 * k) : 0u) | (i + 2 * k + 1 < n ? static_cast<uint32_t>(__ldg(p + 2 * k + 1)) << 16 : 0u);
}

// What a lane has of one row's 32 columns.
template <int TYPE, bool WIDE>
struct Eight {
    float f[TYPE == kTf32 ? 8 : 1];
    uint32_t w[TYPE == kTf32 ? 1 : 4];
    // eight values at a 16-byte boundary
    __device__ __forceinline__ void load_whole(const char *p, bool in, bool half)
    {
        if constexpr (TYPE == kTf32) {
            if (in) load_values<8, WIDE>(f, p, 0, 0, 8, true, half);
            else {
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] = 0.0f;
            }
        } else {
            const uint4 v = in ? __ldg(reinterpret_cast<const uint4 *>(p)) : make_uint4(0u, 0u, 0u, 0u);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        }
    }
    __device__ __forceinline__ void load(const void *base, int64_t row, int i, int n, bool vec, bool half, bool in)
    {
        if constexpr (TYPE == kTf32) {
            if (in) load_values<8, WIDE>(f, base, row, i, n, vec, half);
            else {
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] = 0.0f;
            }
        } else {
            if (in) load_raw<8>(w, base, row, i, n, vec);
            else w[0] = w[1] = w[2] = w[3] = 0u;
        }
    }
};

template <int NR, int TYPE, bool XW, bool WW>
__global__ void __launch_bounds__(kThreads, TYPE == kTf32 ? 1 : 2) shrink_kernel(const LoraArgs a)
{
    constexpr int R8 = 8 * NR;
    extern __shared__ __align__(16) float parts[];           // [warp][row][R8 + 4]
    __shared__ TileList l;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kShrinkRows;
    const int blocks = (a.rank + R8 - 1) / R8, width = blocks * R8;
    const bool x_half = a.x_type == QK_F16, w_half = a.w_type == QK_F16;
    moe::let_next_start();
    moe::wait_for_previous();
    list_adapters(l, a, t0, kShrinkRows);
    for (int j = blockIdx.y; j < l.n; j += gridDim.y) {
        const int id = l.list[j];
        const int64_t a_row = static_cast<int64_t>(id) * a.rank;
        const bool in[2] = {l.ids[g] == id, l.ids[8 + g] == id};
        for (int rb = 0; rb < blocks; ++rb) {
            float acc[NR][4];
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
            struct Turn {
                Eight<TYPE, XW> x[2];
                Eight<TYPE, WW> w[NR];
            };
            // where this lane's values of the warp's first columns are; whole turns need no more than these and their steps
            constexpr int XS = XW ? 4 : 2, WS = WW ? 4 : 2;
            const char *xp = static_cast<const char *>(a.x) + ((t0 + g) * a.ldx + 8 * c) * XS;
            const char *wp = static_cast<const char *>(a.A) + ((a_row + rb * R8 + g) * a.K + 8 * c) * WS;
            const int64_t x_step = 8 * a.ldx * XS, w_step = 8LL * a.K * WS;
            const bool whole = a.vec_x && a.vec_a && rb * R8 + R8 <= a.rank;
            const auto load = [&](Turn &t, int k) {
                if (whole && k + 32 <= a.K) {
                    const char *q = xp + static_cast<int64_t>(k) * XS;
#pragma unroll
                    for (int h = 0; h < 2; ++h, q += x_step) t.x[h].load_whole(q, in[h], x_half);
                    q = wp + static_cast<int64_t>(k) * WS;
#pragma unroll
                    for (int n = 0; n < NR; ++n, q += w_step) t.w[n].load_whole(q, true, w_half);
                    return;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    t.x[h].load(a.x, (t0 + h * 8 + g) * a.ldx, k + 8 * c, a.K, a.vec_x, x_half, in[h] && k < a.K);
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    const int r = rb * R8 + n * 8 + g;
                    t.w[n].load(a.A, (a_row + r) * a.K, k + 8 * c, a.K, a.vec_a, w_half, r < a.rank && k < a.K);
                }
            };
            const auto products = [&](const Turn &t) {
                if constexpr (TYPE == kTf32) {
                    // a turn's products are summed apart: the tensor cores cut a sum at 2^-24 of it, always towards zero
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        float sum[4] = {};
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            const float xa[4] = {t.x[0].f[2 * s], t.x[1].f[2 * s], t.x[0].f[2 * s + 1], t.x[1].f[2 * s + 1]};
                            mma_pieces<XW ? 2 : 1, WW ? 2 : 1>(sum, xa, t.w[n].f[2 * s], t.w[n].f[2 * s + 1]);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[n][i] += sum[i];
                    }
                } else {
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int n = 0; n < NR; ++n)
                            mma16<TYPE>(acc[n], t.x[0].w[2 * s], t.x[1].w[2 * s], t.x[0].w[2 * s + 1], t.x[1].w[2 * s + 1], t.w[n].w[2 * s],
                                        t.w[n].w[2 * s + 1]);
                }
            };
            if constexpr (TYPE == kTf32) {
                for (int k = warp * 32; k < a.K; k += kWarps * 32) {
                    Turn t;
                    load(t, k);
                    products(t);
                }
            } else {
                Turn t[2];
                load(t[0], warp * 32), load(t[1], (warp + kWarps) * 32);
                for (int k = warp * 32; k < a.K; k += 2 * kWarps * 32) {
                    products(t[0]);
                    load(t[0], k + 2 * kWarps * 32);
                    products(t[1]);
                    load(t[1], k + 3 * kWarps * 32);
                }
            }
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<float2 *>(parts + (warp * kShrinkRows + h * 8 + g) * (R8 + 4) + n * 8 + 2 * c) =
                        make_float2(acc[n][2 * h], acc[n][2 * h + 1]);
            __syncthreads();
            const float scale = a.scales ? a.scales[id] : 1.0f;
            for (int i = tid; i < kShrinkRows * R8; i += kThreads) {
                const int row = i / R8, col = i % R8;
                if (l.ids[row] != id) continue;
                float s = parts[row * (R8 + 4) + col];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) s += parts[(w * kShrinkRows + row) * (R8 + 4) + col];
                a.V[(t0 + row) * width + rb * R8 + col] = s * scale;
            }
            __syncthreads();
        }
    }
}

// PIECES: of V, in 16 bits.
template <int NR, int TYPE, int PIECES, bool WW>
__global__ void __launch_bounds__(kThreads, TYPE == kTf32 ? 1 : 2) expand_kernel(const LoraArgs a)
{
    constexpr int R8 = 8 * NR, Q = 2 * NR;                   // ranks of a pass, and of a lane
    __shared__ TileList l;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTallRows;
    const int blocks = (a.rank + R8 - 1) / R8, width = blocks * R8;
    const bool w_half = a.w_type == QK_F16, y_half = a.y_type == QK_F16, y_wide = a.y_type == QK_F32;
    const int n_per = ((a.N + static_cast<int>(gridDim.y) - 1) / static_cast<int>(gridDim.y) + 31) / 32 * 32;
    const int n0 = min(a.N, static_cast<int>(blockIdx.y) * n_per), n1 = min(a.N, n0 + n_per);
    moe::let_next_start();
    moe::wait_for_previous();
    list_adapters(l, a, t0, kTallRows);
    // rows without an adapter
    for (int i = 0; blockIdx.z == 0 && i < kTallRows && t0 + i < a.T; ++i) {
        const bool bad = l.ids[i] >= a.n_adapters;
        if (l.ids[i] >= 0 && !bad) continue;
        if (bad && tid == 0 && blockIdx.y == 0) record_error(a.err, kErrBadIndex);
        if (bad || a.out != a.y)
            for (int n = n0 + tid; n < n1; n += kThreads)
                store_float_as(a.out, (t0 + i) * a.ldo + n, a.y_type,
                               bad ? __int_as_float(0x7fc00000) : load_as_float(a.y, (t0 + i) * a.ldy + n, a.y_type));
    }
    const int m = warp & 1;                                  // the warp's 16 rows, and every fourth 16 columns
    for (int j = blockIdx.z; j < l.n; j += gridDim.z) {
        const int id = l.list[j];
        const int64_t b_row = static_cast<int64_t>(id) * a.N, row0 = t0 + m * 16 + g;
        const bool in[2] = {l.ids[m * 16 + g] == id, l.ids[m * 16 + 8 + g] == id};
        if (!__any_sync(~0u, in[0] || in[1])) continue;
        // V's rows: lane c has its Q ranks of each
        float back[2];
        uint32_t piece[TYPE == kTf32 ? 1 : PIECES][2][TYPE == kTf32 ? 1 : Q / 2];
        float whole[2][TYPE == kTf32 ? Q : 1];
        const auto take = [&](int rb) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float *from = a.V + (row0 + 8 * h) * width + rb * R8 + Q * c;
                float v[Q];
#pragma unroll
                for (int k = 0; k < Q; k += 2) {
                    const float2 f = in[h] ? *reinterpret_cast<const float2 *>(from + k) : make_float2(0.0f, 0.0f);
                    v[k] = f.x, v[k + 1] = f.y;
                }
                back[h] = 1.0f;
                if constexpr (TYPE == kTf32) {
#pragma unroll
                    for (int k = 0; k < Q; ++k) whole[h][k] = v[k];
                } else {
                    float up = 1.0f;
                    if constexpr (TYPE == kF16) {
                        // a power of two puts the row's largest into [2^14, 2^15)
                        uint32_t most = 0;
#pragma unroll
                        for (int k = 0; k < Q; ++k) most = max(most, __float_as_uint(v[k]) & 0x7fffffffu);
                        most = max(most, __shfl_xor_sync(~0u, most, 1)), most = max(most, __shfl_xor_sync(~0u, most, 2));
                        const int ex = most >= 0x7f800000u || most == 0 ? 141 : max(static_cast<int>(most >> 23), 15);
                        up = __uint_as_float(static_cast<uint32_t>(127 + 141 - ex) << 23);
                        back[h] = __uint_as_float(static_cast<uint32_t>(127 - 141 + ex) << 23);
                    }
#pragma unroll
                    for (int k = 0; k < Q; k += 2) {
                        float x = v[k] * up, y = v[k + 1] * up;
#pragma unroll
                        for (int p = 0; p < PIECES; ++p) {
                            const uint32_t w = pack16(x, y, TYPE == kF16);
                            const float2 f = unpack16(w, TYPE == kF16);
                            piece[p][h][k / 2] = w;
                            x -= f.x, y -= f.y;
                        }
                    }
                }
            }
        };
        struct Turn {
            float bf[2][TYPE == kTf32 ? Q : 1];
            uint32_t bw[2][TYPE == kTf32 ? 1 : Q / 2];
            uint4 y[2];                                      // four values: fp32, or two words of 16-bit ones
        };
        // this lane's places in B, y and out
        const int b_col = 4 * (g >> 1) + (g & 1), YS = y_wide ? 4 : 2;
        constexpr int WS = WW ? 4 : 2;
        const char *bp = static_cast<const char *>(a.B) + ((b_row + b_col) * a.rank + Q * c) * WS;
        const char *yp[2] = {static_cast<const char *>(a.y) + (row0 * a.ldy + 4 * c) * YS,
                             static_cast<const char *>(a.y) + ((row0 + 8) * a.ldy + 4 * c) * YS};
        char *op[2] = {static_cast<char *>(a.out) + (row0 * a.ldo + 4 * c) * YS, static_cast<char *>(a.out) + ((row0 + 8) * a.ldo + 4 * c) * YS};
        const bool whole_b = a.vec_b && a.rank % R8 == 0;
        const auto load_b = [&](Turn &t, int n, int rb) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int col = n + b_col + 2 * q;
                if (whole_b && n + 16 <= n1) {
                    const char *p = bp + ((static_cast<int64_t>(n) + 2 * q) * a.rank + rb * R8) * WS;
                    if constexpr (TYPE == kTf32) load_values<Q, WW>(t.bf[q], p, 0, 0, Q, true, w_half);
                    else load_raw<Q>(t.bw[q], p, 0, 0, Q, true);
                } else if constexpr (TYPE == kTf32) {
                    if (col < n1) load_values<Q, WW>(t.bf[q], a.B, (b_row + col) * a.rank, rb * R8 + Q * c, a.rank, a.vec_b, w_half);
                    else {
#pragma unroll
                        for (int i = 0; i < Q; ++i) t.bf[q][i] = 0.0f;
                    }
                } else {
                    if (col < n1) load_raw<Q>(t.bw[q], a.B, (b_row + col) * a.rank, rb * R8 + Q * c, a.rank, a.vec_b);
                    else {
#pragma unroll
                        for (int i = 0; i < Q / 2; ++i) t.bw[q][i] = 0u;
                    }
                }
            }
        };
        const auto load_y = [&](Turn &t, int n) {
            if (!a.vec_y || n + 4 * c + 4 > n1) return;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!in[h]) continue;
                if (y_wide) t.y[h] = *reinterpret_cast<const uint4 *>(yp[h] + 4LL * n);
                else {
                    const uint2 w = *reinterpret_cast<const uint2 *>(yp[h] + 2LL * n);
                    t.y[h].x = w.x, t.y[h].y = w.y;
                }
            }
        };
        if (blocks == 1) take(0);
        Turn next;
        constexpr int kStep = kWarps / 2 * 16;
        int n = n0 + (warp >> 1) * 16;
        if (n < n1) load_b(next, n, 0), load_y(next, n);
        for (; n < n1; n += kStep) {
            Turn t = next;
            if (n + kStep < n1) load_b(next, n + kStep, 0), load_y(next, n + kStep);
            float acc[2][4];
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[q][i] = 0.0f;
            for (int rb = 0; rb < blocks; ++rb) {
                if (blocks > 1) {
                    take(rb);
                    if (rb > 0) load_b(t, n, rb);
                }
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    if constexpr (TYPE == kTf32) {
#pragma unroll
                        for (int s = 0; s < NR; ++s) {
                            const float va[4] = {whole[0][2 * s], whole[1][2 * s], whole[0][2 * s + 1], whole[1][2 * s + 1]};
                            mma_pieces<2, WW ? 2 : 1>(sum, va, t.bf[q][2 * s], t.bf[q][2 * s + 1]);
                        }
                    } else {
#pragma unroll
                        for (int p = PIECES - 1; p >= 0; --p)
#pragma unroll
                            for (int s = 0; s < NR / 2; ++s)
                                mma16<TYPE>(sum, piece[p][0][2 * s], piece[p][1][2 * s], piece[p][0][2 * s + 1], piece[p][1][2 * s + 1],
                                            t.bw[q][2 * s], t.bw[q][2 * s + 1]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[q][i] += sum[i] * back[i >> 1];
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!in[h]) continue;
                const int col = n + 4 * c;
                const float d[4] = {acc[0][2 * h], acc[0][2 * h + 1], acc[1][2 * h], acc[1][2 * h + 1]};
                if (a.vec_y && col + 4 <= n1) {
                    const uint4 w = t.y[h];
                    if (y_wide) {
                        *reinterpret_cast<float4 *>(op[h] + 4LL * n) = make_float4(
                            __uint_as_float(w.x) + d[0], __uint_as_float(w.y) + d[1], __uint_as_float(w.z) + d[2], __uint_as_float(w.w) + d[3]);
                    } else {
                        const float2 f0 = unpack16(w.x, y_half), f1 = unpack16(w.y, y_half);
                        *reinterpret_cast<uint2 *>(op[h] + 2LL * n) =
                            make_uint2(pack16(f0.x + d[0], f0.y + d[1], y_half), pack16(f1.x + d[2], f1.y + d[3], y_half));
                    }
                } else {
                    const int64_t row = row0 + 8 * h;
                    for (int i = 0; i < 4 && col + i < n1; ++i)
                        store_float_as(a.out, row * a.ldo + col + i, a.y_type, load_as_float(a.y, row * a.ldy + col + i, a.y_type) + d[i]);
                }
            }
        }
    }
}

__device__ __forceinline__ void lora_copy16(uint32_t dst, const void *src, bool on)
{
    if (on) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lora_lds(uint32_t p)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
    return v;
}

// The same for 16-bit adapters, and activations of any type, in whole vectors (rows of x, A, B, y and out on 16 bytes, K, N and the rank
// multiples of 8), which leaves every 16 bytes either inside their row or outside, and so no other path.  A warp's
// operands come through a ring of its own, two turns ahead.
constexpr int kTurns = 3;                                    // of a warp on their way or at work

__host__ __device__ constexpr int shrink_turn_bytes(int NR, bool XW) { return kTallRows * (XW ? 128 : 64) + 8 * NR * 64; }

// TYPE: that of x and A; kTf32 where x is fp32 (XW) or the other 16-bit type.
template <int NR, int TYPE, bool XW>
__global__ void __launch_bounds__(kThreads, 1) shrink16_kernel(const LoraArgs a)
{
    constexpr int R8 = 8 * NR, XP = XW ? 128 : 64, XC = XP / 16, TURN = shrink_turn_bytes(NR, XW);
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ TileList l;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTallRows;
    const uint32_t mine = smem_u32(ring) + warp * kTurns * TURN;
    float *parts = reinterpret_cast<float *>(ring);          // afterwards: [warp][row][R8 + 4]
    const bool x_half = a.x_type == QK_F16, w_half = a.w_type == QK_F16;
    const int width = (a.rank + R8 - 1) / R8 * R8;
    moe::let_next_start();
    moe::wait_for_previous();
    list_adapters(l, a, t0, kTallRows);
    for (int j = blockIdx.y; j < l.n; j += gridDim.y) {
        const int id = l.list[j];
        const float scale = a.scales ? a.scales[id] : 1.0f;
        // a lane copies 16 bytes of every eighth row of A, and of every (32 / XC)th of x; and reads every eighth
        const int x_row = lane / XC, x_ch = lane % XC;
        unsigned rows = 0, copied = 0;
#pragma unroll
        for (int i = 0; i < kTallRows / 8; ++i) rows |= (l.ids[8 * i + g] == id) << i;
#pragma unroll
        for (int i = 0; i < XC; ++i) copied |= (l.ids[i * (32 / XC) + x_row] == id) << i;
        const char *x0 = static_cast<const char *>(a.x) + (t0 + x_row) * a.ldx * (XW ? 4 : 2) + 16 * x_ch;
        // (of fp32, the 16-byte pieces of odd rows lie exchanged: no bank conflicts when two rows are read at once)
        const uint32_t x_to = x_row * XP + 16 * (XW ? x_ch ^ (x_row & 1) : x_ch);
        for (int rb = 0; rb * R8 < a.rank; ++rb) {
            const uint16_t *w0 = static_cast<const uint16_t *>(a.A) + (static_cast<int64_t>(id) * a.rank + rb * R8 + g) * a.K + 8 * c;
            const int tiles = min(NR, (a.rank - rb * R8) / 8);
            const int64_t x_step = (32 / XC) * a.ldx * (XW ? 4 : 2), w_step = 8LL * a.K;
            const auto fetch = [&](int k, int slot) {
                if (k < a.K) {
                    // past the rows' end: zeros
                    uint32_t to = mine + slot * TURN + x_to;
                    if (k + x_ch * (XW ? 4 : 8) < a.K) {
                        const char *q = x0 + static_cast<int64_t>(k) * (XW ? 4 : 2);
#pragma unroll
                        for (int i = 0; i < XC; ++i, q += x_step) lora_copy16(to + i * 512, q, (copied >> i) & 1u);
                    } else {
#pragma unroll
                        for (int i = 0; i < XC; ++i) asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(to + i * 512), "r"(0) : "memory");
                    }
                    to = mine + slot * TURN + kTallRows * XP + g * 64 + 16 * c;
                    if (k + 8 * c < a.K) {
                        const uint16_t *q = w0 + k;
#pragma unroll
                        for (int i = 0; i < NR; ++i, q += w_step) lora_copy16(to + i * 512, q, i < tiles);
                    } else {
#pragma unroll
                        for (int i = 0; i < NR; ++i) asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(to + i * 512), "r"(0) : "memory");
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            constexpr int kTurn = kWarps * 32;
            int k = warp * 32;
#pragma unroll
            for (int i = 0; i < kTurns - 1; ++i) fetch(k + i * kTurn, i);
            float acc[2][NR][4];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            for (int slot = 0; k < a.K; k += kTurn) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kTurns - 2) : "memory");
                __syncwarp();                                // this turn has landed, and the slot before it is free
                fetch(k + (kTurns - 1) * kTurn, slot == 0 ? kTurns - 1 : slot - 1);
                const uint32_t at = mine + slot * TURN;
                // (rows of other tokens hold what they held; ranks past the last are dropped below)
                uint4 x[2][2][XW ? 2 : 1], w[NR];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int q = 0; q < (XW ? 2 : 1); ++q) {
                            x[m][h][q] = lora_lds(at + (16 * m + 8 * h + g) * XP + 16 * (XW ? (2 * c + q) ^ (g & 1) : c));
                            if (!((rows >> (2 * m + h)) & 1u)) x[m][h][q] = zero;
                        }
#pragma unroll
                for (int n = 0; n < NR; ++n) w[n] = lora_lds(at + kTallRows * XP + n * 512 + g * 64 + 16 * c);
                if constexpr (TYPE != kTf32) {
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const uint4 p = x[m][0][0], q = x[m][1][0];
                            mma16<TYPE>(acc[m][n], p.x, q.x, p.y, q.y, w[n].x, w[n].y);
                        }
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            const uint4 p = x[m][0][0], q = x[m][1][0];
                            mma16<TYPE>(acc[m][n], p.z, q.z, p.w, q.w, w[n].z, w[n].w);
                        }
                } else {
                    // (summed apart by turns, as above)
                    float2 v[4][2][2];                       // a lane's columns 2s and 2s + 1
#pragma unroll
                    for (int s = 0; s < 4; ++s)
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint4 p = x[m][h][XW ? s / 2 : 0];
                                if constexpr (XW)
                                    v[s][m][h] = s % 2 ? make_float2(__uint_as_float(p.z), __uint_as_float(p.w)) : make_float2(__uint_as_float(p.x), __uint_as_float(p.y));
                                else
                                    v[s][m][h] = unpack16(s == 0 ? p.x : s == 1 ? p.y : s == 2 ? p.z : p.w, x_half);
                            }
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        float sum[2][4] = {};
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            const float2 b = unpack16(s == 0 ? w[n].x : s == 1 ? w[n].y : s == 2 ? w[n].z : w[n].w, w_half);
#pragma unroll
                            for (int m = 0; m < 2; ++m) {
                                const float p[4] = {v[s][m][0].x, v[s][m][1].x, v[s][m][0].y, v[s][m][1].y};
                                mma_pieces<XW ? 2 : 1, 1>(sum[m], p, b.x, b.y);
                            }
                        }
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[m][n][i] += sum[m][i];
                    }
                }
                slot = slot + 1 == kTurns ? 0 : slot + 1;
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        *reinterpret_cast<float2 *>(parts + (warp * kTallRows + m * 16 + h * 8 + g) * (R8 + 4) + n * 8 + 2 * c) =
                            make_float2(acc[m][n][2 * h], acc[m][n][2 * h + 1]);
            __syncthreads();
            for (int i = tid * 4; i < kTallRows * R8; i += kThreads * 4) {
                const int r = i / R8, col = i % R8;
                float4 s = *reinterpret_cast<const float4 *>(parts + r * (R8 + 4) + col);
#pragma unroll
                for (int v = 1; v < kWarps; ++v) {
                    const float4 p = *reinterpret_cast<const float4 *>(parts + (v * kTallRows + r) * (R8 + 4) + col);
                    s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
                }
                if (l.ids[r] == id)
                    *reinterpret_cast<float4 *>(a.V + (t0 + r) * width + rb * R8 + col) =
                        rb * R8 + col < a.rank ? make_float4(s.x * scale, s.y * scale, s.z * scale, s.w * scale) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            __syncthreads();
        }
    }
}

// A warp's turn is 32 columns: B's 32 rows, in a pitch that keeps two rows' 16 bytes apart, and the tile's 32 rows of y.
__host__ __device__ constexpr int expand_turn_bytes(int NR, int ys) { return 32 * (16 * NR + 16) + 32 * 32 * ys; }

// Ranks up to 8 NR in one pass.
template <int NR, int TYPE, int PIECES, bool YW>
__global__ void __launch_bounds__(kThreads, 1) expand16_kernel(const LoraArgs a)
{
    constexpr int Q = 2 * NR, PITCH = 16 * NR + 16, YS = YW ? 4 : 2, TURN = expand_turn_bytes(NR, YS), YP = 32 * YS;
    constexpr int BL = NR, YL = YP / 16;                     // 16-byte pieces of a row of B (2 NR bytes a lane of 8), and of y
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ TileList l;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTallRows;
    const bool y_half = a.y_type == QK_F16;
    const int turns_all = (a.N + 31) / 32, per = (turns_all + static_cast<int>(gridDim.y) - 1) / static_cast<int>(gridDim.y);
    const int first = min(turns_all, static_cast<int>(blockIdx.y) * per), last = min(turns_all, first + per);
    const uint32_t mine = smem_u32(ring) + warp * kTurns * TURN;
    moe::let_next_start();
    moe::wait_for_previous();
    list_adapters(l, a, t0, kTallRows);
    // rows without an adapter
    unsigned none = __ballot_sync(~0u, blockIdx.z == 0 && t0 + lane < a.T && (l.ids[lane] < 0 || l.ids[lane] >= a.n_adapters));
    for (; none; none &= none - 1) {
        const int i = __ffs(none) - 1;
        const bool bad = l.ids[i] >= 0;
        if (bad && tid == 0 && blockIdx.y == 0) record_error(a.err, kErrBadIndex);
        if (bad || a.out != a.y)
            for (int n = 32 * first + tid; n < min(a.N, 32 * last); n += kThreads)
                store_float_as(a.out, (t0 + i) * a.ldo + n, a.y_type,
                               bad ? __int_as_float(0x7fc00000) : load_as_float(a.y, (t0 + i) * a.ldy + n, a.y_type));
    }
    for (int j = blockIdx.z; j < l.n; j += gridDim.z) {
        const int id = l.list[j];
        // a lane copies 16 bytes of every (32 / BL)th row of B, and of every (32 / YL)th of y
        const int b_row = lane / BL, b_ch = lane % BL, y_row = lane / YL, y_ch = lane % YL;
        const bool b_on = 8 * b_ch < a.rank;
        unsigned rows = 0;
#pragma unroll
        for (int i = 0; i < YL; ++i) rows |= (l.ids[i * (32 / YL) + y_row] == id) << i;
        int from = first + warp;                             // the turn that is fetched next
        const uint16_t *B = static_cast<const uint16_t *>(a.B) + (static_cast<int64_t>(id) * a.N + 32 * from + b_row) * a.rank + 8 * b_ch;
        const char *Y = static_cast<const char *>(a.y) + ((t0 + y_row) * a.ldy + 32 * from) * YS + 16 * y_ch;
        const int64_t b_step = (32 / BL) * static_cast<int64_t>(a.rank), y_step = (32 / YL) * a.ldy * YS;
        const auto fetch = [&](int slot) {
            if (from < last) {
                const uint32_t to = mine + slot * TURN;
                const uint16_t *b = B;
#pragma unroll
                for (int i = 0; i < BL; ++i, b += b_step)
                    lora_copy16(to + (i * (32 / BL) + b_row) * PITCH + 16 * b_ch, b, b_on && 32 * from + i * (32 / BL) + b_row < a.N);
                const char *y = Y;
                const bool y_on = 32 * from + y_ch * (16 / YS) < a.N;
#pragma unroll
                for (int i = 0; i < YL; ++i, y += y_step)
                    lora_copy16(to + 32 * PITCH + (i * (32 / YL) + y_row) * YP + 16 * y_ch, y, y_on && (rows >> i) & 1u);
                from += kWarps, B += kWarps * 32 * static_cast<int64_t>(a.rank), Y += kWarps * 32 * YS;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        if (a.rank < 8 * NR) {
            // ranks past the last hold zeros for good
            for (int i = lane; i < kTurns * 32 * NR; i += 32) {
                const int ch = i % NR, row = i / NR % 32, slot = i / NR / 32;
                if (8 * ch >= a.rank)
                    *reinterpret_cast<uint4 *>(ring + warp * kTurns * TURN + slot * TURN + row * PITCH + 16 * ch) = make_uint4(0u, 0u, 0u, 0u);
            }
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < kTurns - 1; ++i) fetch(i);
        bool in[2][2];
        float back[2][2];
        uint32_t piece[PIECES][2][2][Q / 2];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                in[m][h] = l.ids[m * 16 + h * 8 + g] == id;
                const float *from = a.V + (t0 + m * 16 + h * 8 + g) * (8 * NR) + Q * c;
                float v[Q], up = 1.0f;
#pragma unroll
                for (int k = 0; k < Q; k += 4) {
                    const float4 f = in[m][h] ? *reinterpret_cast<const float4 *>(from + k) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    v[k] = f.x, v[k + 1] = f.y, v[k + 2] = f.z, v[k + 3] = f.w;
                }
                back[m][h] = 1.0f;
                if constexpr (TYPE == kF16) {
                    // a power of two puts the row's largest into [2^14, 2^15)
                    uint32_t most = 0;
#pragma unroll
                    for (int k = 0; k < Q; ++k) most = max(most, __float_as_uint(v[k]) & 0x7fffffffu);
                    most = max(most, __shfl_xor_sync(~0u, most, 1)), most = max(most, __shfl_xor_sync(~0u, most, 2));
                    const int ex = most >= 0x7f800000u || most == 0 ? 141 : max(static_cast<int>(most >> 23), 15);
                    up = __uint_as_float(static_cast<uint32_t>(127 + 141 - ex) << 23);
                    back[m][h] = __uint_as_float(static_cast<uint32_t>(127 - 141 + ex) << 23);
                }
#pragma unroll
                for (int k = 0; k < Q; k += 2) {
                    float x = v[k] * up, y = v[k + 1] * up;
#pragma unroll
                    for (int p = 0; p < PIECES; ++p) {
                        const uint32_t w = pack16(x, y, TYPE == kF16);
                        const float2 f = unpack16(w, TYPE == kF16);
                        piece[p][m][h][k / 2] = w;
                        x -= f.x, y -= f.y;
                    }
                }
            }
        int slot = 0;
        for (int turn = first + warp; turn < last; turn += kWarps) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kTurns - 2) : "memory");
            __syncwarp();                                    // this turn has landed, and the slot before it is free
            fetch(slot == 0 ? kTurns - 1 : slot - 1);
            const uint32_t at = mine + slot * TURN;
            float sum[2][4][4];
            uint32_t w[4][Q / 2];
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                const uint32_t from = at + (8 * (g >> 1) + 2 * nt + (g & 1)) * PITCH + 2 * Q * c;
                if constexpr (Q >= 8) {
#pragma unroll
                    for (int k = 0; k < Q / 8; ++k) {
                        const uint4 v = lora_lds(from + 16 * k);
                        w[nt][4 * k] = v.x, w[nt][4 * k + 1] = v.y, w[nt][4 * k + 2] = v.z, w[nt][4 * k + 3] = v.w;
                    }
                } else {
                    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[nt][0]), "=r"(w[nt][1]) : "r"(from));
                }
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int k = 0; k < 4; ++k) sum[m][nt][k] = 0.0f;
            }
            // eight sums in turn: a product waits for the one before it in its own
#pragma unroll
            for (int p = PIECES - 1; p >= 0; --p)
#pragma unroll
                for (int s = 0; s < NR / 2; ++s)
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                        for (int m = 0; m < 2; ++m)
                            mma16<TYPE>(sum[m][nt], piece[p][m][0][2 * s], piece[p][m][1][2 * s], piece[p][m][0][2 * s + 1],
                                        piece[p][m][1][2 * s + 1], w[nt][2 * s], w[nt][2 * s + 1]);
            const int col = turn * 32 + 8 * c;
            char *out0 = static_cast<char *>(a.out) + ((t0 + g) * a.ldo + col) * YS;
            const int64_t o_step = 8 * a.ldo * YS;
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = m * 16 + h * 8 + g;
                    float d[8];
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt) d[2 * nt] = sum[m][nt][2 * h], d[2 * nt + 1] = sum[m][nt][2 * h + 1];
                    if constexpr (TYPE == kF16) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) d[k] *= back[m][h];
                    }
                    char *out = out0 + (2 * m + h) * o_step;
                    const bool on = in[m][h] && col < a.N;
                    if constexpr (YW) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint4 v = lora_lds(at + 32 * PITCH + row * YP + 32 * c + 16 * k);
                            if (on)
                                *(reinterpret_cast<float4 *>(out) + k) = make_float4(__uint_as_float(v.x) + d[4 * k], __uint_as_float(v.y) + d[4 * k + 1],
                                                                                     __uint_as_float(v.z) + d[4 * k + 2], __uint_as_float(v.w) + d[4 * k + 3]);
                        }
                    } else {
                        const uint4 v = lora_lds(at + 32 * PITCH + row * YP + 16 * c);
                        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
                        uint32_t r[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 f = unpack16(u[k], y_half);
                            r[k] = pack16(f.x + d[2 * k], f.y + d[2 * k + 1], y_half);
                        }
                        if (on) *reinterpret_cast<uint4 *>(out) = make_uint4(r[0], r[1], r[2], r[3]);
                    }
                }
            slot = slot + 1 == kTurns ? 0 : slot + 1;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();
    }
}

// 16-bit adapters in whole vectors, ranks of one pass.
bool ring_ok(const LoraArgs &a)
{
    return a.w_type != QK_F32 && a.vec_x && a.vec_a && a.vec_b && a.vec_y && a.N % 8 == 0 && a.rank <= kBlockRank;
}

// A tile's adapters are shared out over blocks, at least two: with one, a tile at the border of two requests takes twice
// as long as the others, and the launch with it (4096 tokens of 7 requests: 35 and 55 us).  But a block that finds no
// adapter for itself costs its start, so that the launch's blocks are two rounds of the GPU at most (493 tokens of 34
// requests, rank 64: 39 us, 52 with all 32 that a tile's tokens can have).  Many tokens whose neighbours differ pay for it:
// each adapter of a tile is a pass of a block (4096 tokens of 7 requests one after another 57 us, alternating over 8 adapters
// 329, over 64 1207).
unsigned share_of(const LoraArgs &a, unsigned blocks, int sms)
{
    return std::min(static_cast<unsigned>(std::min<int64_t>(kTallRows, a.n_adapters)), std::max(2u, 2u * sms / blocks));
}

// TYPE: of the adapters.
template <int NR, int TYPE, int PIECES, bool YW>
cudaError_t launch_ring(const LoraArgs &a, int sms, cudaStream_t st)
{
    const bool wide = a.x_type == QK_F32;
    const auto shrink = a.x_type == a.w_type ? shrink16_kernel<NR, TYPE, false> : wide ? shrink16_kernel<NR, kTf32, true> : shrink16_kernel<NR, kTf32, false>;
    const auto expand = expand16_kernel<NR, TYPE, PIECES, YW>;
    constexpr int sums = static_cast<int>(sizeof(float)) * kWarps * kTallRows * (8 * NR + 4);
    const int smem = std::max(sums, kWarps * kTurns * shrink_turn_bytes(NR, wide)), ring = kWarps * kTurns * expand_turn_bytes(NR, YW ? 4 : 2);
    cudaError_t e = cudaFuncSetAttribute(shrink, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(expand, cudaFuncAttributeMaxDynamicSharedMemorySize, ring);
    if (e != cudaSuccess) return e;
    const unsigned tiles = static_cast<unsigned>((a.T + kTallRows - 1) / kTallRows);
    e = moe::launch_chained(shrink, dim3(tiles, share_of(a, tiles, sms)), kThreads, smem, st, library_programmatic(), a);
    if (e != cudaSuccess) return e;
    // columns are cut where tiles do not fill the GPU, down to a turn a warp
    const unsigned cuts = static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>((a.N + 32 * kWarps - 1) / (32 * kWarps), sms / tiles)));
    return moe::launch_chained(expand, dim3(tiles, cuts, share_of(a, tiles * cuts, sms)), kThreads, ring, st, true, a);
}

// SHRINK, EXPAND: the launches' types.
template <int NR, int SHRINK, int EXPAND, int PIECES, bool XW, bool WW>
cudaError_t launch_tall_as(const LoraArgs &a, int sms, cudaStream_t st)
{
    constexpr int R8 = 8 * NR;
    const int smem = static_cast<int>(sizeof(float)) * kWarps * kShrinkRows * (R8 + 4);
    const auto shrink = shrink_kernel<NR, SHRINK, XW, WW>;
    cudaError_t e = cudaFuncSetAttribute(shrink, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const unsigned tiles = static_cast<unsigned>((a.T + kTallRows - 1) / kTallRows);
    const unsigned halves = static_cast<unsigned>((a.T + kShrinkRows - 1) / kShrinkRows);
    e = moe::launch_chained(shrink, dim3(halves, share_of(a, halves, sms)), kThreads, smem, st, library_programmatic(), a);
    if (e != cudaSuccess) return e;
    // columns are cut where tiles do not fill the GPU, down to two turns
    const unsigned cuts = static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>((a.N + 127) / 128, sms / tiles)));
    return moe::launch_chained(expand_kernel<NR, EXPAND, PIECES, WW>, dim3(tiles, cuts, share_of(a, tiles * cuts, sms)), kThreads, 0, st, true, a);
}

template <int NR, int TYPE, int PIECES, bool YW>
cudaError_t launch_w16(const LoraArgs &a, int sms, cudaStream_t st)
{
    if (ring_ok(a)) return launch_ring<NR, TYPE, PIECES, YW>(a, sms, st);
    if (a.x_type == a.w_type) return launch_tall_as<NR, TYPE, TYPE, PIECES, false, false>(a, sms, st);
    return a.x_type == QK_F32 ? launch_tall_as<NR, kTf32, TYPE, PIECES, true, false>(a, sms, st)
                              : launch_tall_as<NR, kTf32, TYPE, PIECES, false, false>(a, sms, st);
}

template <int NR>
cudaError_t launch_tall_types(const LoraArgs &a, int sms, cudaStream_t st)
{
    // 16-bit adapters: the same products in the same order by rings or through registers, so that bits depend on no alignment
    if (a.w_type == QK_F16) return a.y_type == QK_F32 ? launch_w16<NR, kF16, 2, true>(a, sms, st) : launch_w16<NR, kF16, 2, false>(a, sms, st);
    if (a.w_type == QK_BF16)
        return a.y_type == QK_F32   ? launch_w16<NR, kBf16, 3, true>(a, sms, st)
               : a.y_type == QK_F16 ? launch_w16<NR, kBf16, 3, false>(a, sms, st)
                                    : launch_w16<NR, kBf16, 2, false>(a, sms, st);
    return a.x_type == QK_F32 ? launch_tall_as<NR, kTf32, kTf32, 2, true, true>(a, sms, st) : launch_tall_as<NR, kTf32, kTf32, 2, false, true>(a, sms, st);
}

int tall_blocks(int rank) { return rank <= 16 ? 2 : rank <= 32 ? 4 : 8; }      // 8-rank tiles of a pass

cudaError_t launch_tall(const LoraArgs &a, int sms, cudaStream_t st)
{
    switch (tall_blocks(a.rank)) {
    case 2: return launch_tall_types<2>(a, sms, st);
    case 4: return launch_tall_types<4>(a, sms, st);
    default: return launch_tall_types<8>(a, sms, st);
    }
}

template <int MT, int NR>
cudaError_t launch_types(const LoraArgs &a, cudaStream_t st)
{
    if (a.x_type == QK_F32)
        return a.w_type == QK_F32 ? launch_as<MT, NR, true, true>(a, st) : launch_as<MT, NR, true, false>(a, st);
    return a.w_type == QK_F32 ? launch_as<MT, NR, false, true>(a, st) : launch_as<MT, NR, false, false>(a, st);
}

template <int MT>
cudaError_t launch_rank(const LoraArgs &a, cudaStream_t st)
{
    if (a.rank <= 8) return launch_types<MT, 1>(a, st);
    if (a.rank <= 16) return launch_types<MT, 2>(a, st);
    if (a.rank <= 32) return launch_types<MT, 4>(a, st);
    return launch_types<MT, 8>(a, st);
}

bool multiple(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool type_ok(int t) { return t == QK_F32 || t == QK_F16 || t == QK_BF16; }
int size_of(int t) { return t == QK_F32 ? 4 : 2; }

}  // namespace
}  // namespace qk

using namespace qk;

namespace {
// Which calls with a workspace take the two-launch form.  K = N = 4096, bf16 adapters, calls one after another in a graph (what
// they read is in L2), two launches and one.  bf16 activations of rank 16: one token 7.8 us and 6.3, 23 of 23 adapters 9.8 and
// 10.5, 64 of 48 13.0 and 20.6 (of 4 11.1 and 9.4); rank 64: one token 17.0 and 11.8, 23 22.1 and 32.4, 64 30.7 and 79.8.  fp32
// activations of rank 16: 64 of 48 25.4 and 20.6; of rank 64 52.9 and 81.2 (of 4 38.1 and 18.3).  Which adapters a call has is
// not known here; with caches emptied between calls one token of rank 64 took 23.7 and 25.8.  Adapters in fp32 and ranks past
// one pass: many tokens only.
bool two_launches(int64_t T, int rank, int x_type, int w_type)
{
    if (T >= 256) return true;
    if (w_type == QK_F32 || rank > kBlockRank) return false;
    return x_type != QK_F32 ? T > 16 || rank > 16 : T >= 16 && rank > 32;
}
size_t lora_bytes(int64_t T, int rank)
{
    const int r8 = 8 * tall_blocks(rank);
    return static_cast<size_t>(T) * ((rank + r8 - 1) / r8 * r8) * sizeof(float);
}
}  // namespace

extern "C" size_t qk_lora_workspace_bytes(int64_t T, int rank)
{
    return T <= 0 || T > (1 << 26) || rank <= 0 || rank > kMaxRank ? 0 : lora_bytes(T, rank);
}

extern "C" int qk_lora(const void *x, int64_t ldx, int x_type, int64_t T, int64_t K, const void *A, const void *B, int w_type,
                       int64_t n_adapters, int rank, int64_t N, const int32_t *ids, const float *scales, const void *y,
                       int64_t ldy, void *out, int64_t ldo, int y_type, void *workspace,
                       size_t workspace_bytes, qk_stream_t stream)
{
    if (!type_ok(x_type) || !type_ok(w_type) || !type_ok(y_type)) return QK_ERR_TYPE;
    if (T < 0 || K <= 0 || N <= 0 || n_adapters <= 0 || rank <= 0) return QK_ERR_BAD_DIM;
    if (ldx == 0) ldx = K;
    if (ldy == 0) ldy = N;
    if (ldo == 0) ldo = N;
    if (ldx < K || ldy < N || ldo < N || (out && out == y && T > 1 && ldo != ldy)) return QK_ERR_BAD_DIM;
    if (rank > kMaxRank || K > (1 << 24) || N > (1 << 24) || T > (1 << 26) || n_adapters > INT32_MAX) return QK_ERR_TOO_LARGE;
    if (T == 0) return QK_OK;
    if (!x || !A || !B || !ids || !y || !out) return QK_ERR_NULL;
    if (!multiple(x, size_of(x_type)) || !multiple(A, size_of(w_type)) || !multiple(B, size_of(w_type)) ||
        !multiple(y, size_of(y_type)) || !multiple(out, size_of(y_type)) || !multiple(ids, 4) || !multiple(scales, 4))
        return QK_ERR_ALIGN;
    LoraArgs a{};
    a.x = x, a.y = y, a.A = A, a.B = B, a.out = out, a.ldx = ldx, a.ldy = ldy, a.ldo = ldo, a.T = T;
    a.n_adapters = n_adapters, a.x_type = x_type, a.y_type = y_type, a.w_type = w_type;
    a.K = static_cast<int>(K), a.N = static_cast<int>(N), a.rank = rank, a.ids = ids, a.scales = scales;
    // rows that start on 16 bytes
    const auto rows_ok = [](const void *p, int64_t ld, int size, int n) { return multiple(p, n * size) && ld % n == 0; };
    a.vec_x = rows_ok(x, ldx, size_of(x_type), 16 / size_of(x_type));
    a.vec_a = rows_ok(A, K, size_of(w_type), 16 / size_of(w_type));
    a.vec_b = rows_ok(B, rank, size_of(w_type), 16 / size_of(w_type));
    a.vec_y = rows_ok(y, ldy, size_of(y_type), 16 / size_of(y_type)) && rows_ok(out, ldo, size_of(y_type), 16 / size_of(y_type));
    a.err = library_error_word();
    int sms = 0, smem = 0;
    if (!a.err || !device_limits(&sms, &smem)) return QK_ERR_CUDA;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (workspace && !multiple(workspace, 256)) return QK_ERR_WORKSPACE;
    if (two_launches(T, rank, x_type, w_type) && workspace && workspace_bytes >= lora_bytes(T, rank)) {
        a.V = static_cast<float *>(workspace);
        return launch_tall(a, sms, st) == cudaSuccess ? QK_OK : QK_ERR_CUDA;
    }
    // few tokens may each have an adapter of their own: as many clusters a tile as the GPU holds, up to its tokens
    const bool tall = T > 16LL * sms / kCluster;
    const int rows = tall ? 32 : 16;
    const int64_t tiles = (T + rows - 1) / rows;
    a.steps = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({rows, n_adapters, T, 4LL * sms / (kCluster * tiles)})));
    // what is left of the GPU takes a part of the columns each, down to a turn a warp, and forms A x for itself
    a.cuts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((a.N + 16 * kWarps * kCluster - 1) / (16 * kWarps * kCluster),
                                                                      (rank <= 16 ? 2 : 1) * sms / (kCluster * tiles * a.steps))));
    const cudaError_t e = tall ? launch_rank<2>(a, st) : launch_rank<1>(a, st);
    return e == cudaSuccess ? QK_OK : QK_ERR_CUDA;
}
