// qk_moe.cu -- the experts' feed-forward products: the entry point, its
// argument checks, and the kernels around the products (the plan that groups
// assignments by expert, the operands' layout, the weighted sum).
#include <algorithm>
#include <atomic>

#include "qk_moe.cuh"
#include "qk_tc.cuh"

namespace qk {
using namespace moe;
namespace {

constexpr int kPlanThreads = 1024;
// Tokens an expert from which the tile form takes them (qk_moe_tile.cuh).
constexpr int kTileFrom = 16;
std::atomic<int> g_skip_chunk{-1};

struct PlanArgs {
    const int32_t *ids;
    int n, experts, per_warp;      // per_warp: ids of a warp, a multiple of 32
    int tile_from, tile_tokens;    // tokens of an expert that goes by tile sets, and of a set at most
    Plan plan;
    int *err;
};

__device__ __forceinline__ int4 plus(int4 a, int4 b) { return make_int4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }

// Sums over the threads before this one, and over all of the thread block.
__device__ __forceinline__ int4 scan_before(const int4 v, int4 *warp_sums, int4 &all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const auto scan = [&](int4 in) {
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int4 o = make_int4(__shfl_up_sync(~0u, in.x, d), __shfl_up_sync(~0u, in.y, d), __shfl_up_sync(~0u, in.z, d),
                                     __shfl_up_sync(~0u, in.w, d));
            if (lane >= d) in = plus(in, o);
        }
        return in;
    };
    const auto of_lane = [&](int4 in, int from) {
        return make_int4(__shfl_sync(~0u, in.x, from), __shfl_sync(~0u, in.y, from), __shfl_sync(~0u, in.z, from),
                         __shfl_sync(~0u, in.w, from));
    };
    const int4 in = scan(v);
    if (lane == 31) warp_sums[warp] = in;
    __syncthreads();
    const int4 sums = scan(warp_sums[lane]);                 // kPlanThreads / 32 warps: one a lane
    all = of_lane(sums, 31);
    const int4 before = of_lane(sums, warp > 0 ? warp - 1 : 0);
    const int4 mine = make_int4(in.x - v.x, in.y - v.y, in.z - v.z, in.w - v.w);
    return warp > 0 ? plus(before, mine) : mine;
}

// Groups the assignments by expert: a counting sort.  Each warp counts its own run of ids, a thread an expert turns the
// counts into first places, and each warp places its run again in order, so that places rise with the assignments.
// Many ids are shared out over the blocks of a cluster, which read each other's counts.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a)
{
    extern __shared__ int counts[];             // [warp][expert]
    __shared__ int4 warp_sums[kPlanThreads / 32];
    __shared__ int block_count[kMaxExperts], place_of[kMaxExperts], octet_of[kMaxExperts];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int blocks = static_cast<int>(gridDim.x), rank = static_cast<int>(blockIdx.x);
    const int64_t first = (static_cast<int64_t>(rank) * (kPlanThreads / 32) + warp) * a.per_warp;
    const int64_t last = min(static_cast<int64_t>(a.n), first + a.per_warp);
    const int warps = min(kPlanThreads / 32, (a.n + a.per_warp - 1) / a.per_warp);      // that may have ids
    let_next_start();
    for (int i = threadIdx.x; i < warps * a.experts; i += kPlanThreads) counts[i] = 0;
    __syncthreads();
    wait_for_previous();
    int *mine = counts + warp * a.experts;
    constexpr int kAhead = 4;                   // loads on their way at once
    // f(assignment, id, the lanes with the same live id) over this warp's run, in order; -1: no live id
    const auto over_run = [&](auto f) {
        for (int64_t base = first; base < last; base += 32 * kAhead) {
            int id[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) id[k] = base + 32 * k + lane < last ? a.ids[base + 32 * k + lane] : -1;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (base + 32 * k >= last) break;
                const bool live = id[k] >= 0 && id[k] < a.experts;
                f(base + 32 * k + lane, id[k], live, __match_any_sync(~0u, live ? id[k] : -1));
                __syncwarp();
            }
        }
    };
    over_run([&](int64_t, int id, bool live, unsigned same) {
        if (id >= a.experts) record_error(a.err, kErrBadIndex);
        if (live && lane == __ffs(same) - 1) mine[id] += __popc(same);
    });
    __syncthreads();
    const int e = threadIdx.x;
    int n = 0;
    if (e < a.experts) {
        for (int w = 0; w < warps; ++w) {
            const int k = counts[w * a.experts + e];
            counts[w * a.experts + e] = n;
            n += k;
        }
        block_count[e] = n;
    }
    int before = 0;                             // the expert's ids in the blocks before
    if (blocks > 1) {
        cluster_sync();
        if (e < a.experts) {
            n = 0;
            for (int q = 0; q < blocks; ++q) {
                int k;
                asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(k) : "r"(mapa_shared(smem_u32(block_count + e), q)));
                if (q < rank) before += k;
                n += k;
            }
        }
    }
    // Which form takes which experts.  Those of 16 tokens or more suit the many-token form (512 tokens of 8 of 128 experts
    // take 291 us in a graph, as from 8 tokens; from 48 349).  But where they would add few sets to those of the
    // few-token form it takes them, too, and where that one would have few of its own the other takes all: a launch that
    // does not fill the GPU costs more than they do (64 tokens: 27 + 15 us for seven experts).
    constexpr int kRowTokens = 8 * kSetOctets;
    const int parts = (n + a.tile_tokens - 1) / a.tile_tokens;
    // tile sets as even as 32 tokens allow, none of them empty
    const int per = n > 0 ? ((n + parts - 1) / parts + 31) / 32 * 32 : 1, tile_n = (n + per - 1) / per;
    const bool many = n >= a.tile_from;
    const int row_sets = (n + kRowTokens - 1) / kRowTokens;
    int4 sum;
    scan_before(make_int4(many ? 0 : row_sets, many ? row_sets : 0, many ? tile_n : 0, 0), warp_sums, sum);
    __syncthreads();
    const bool tiled = sum.y <= sum.x / 4 ? false : 2 * sum.x <= sum.z ? n > 0 : many;
    const int rows_n = tiled ? 0 : n;
    int4 all;
    const int4 at = scan_before(make_int4(n, (rows_n + 7) / 8, tiled ? 0 : row_sets, tiled ? tile_n : 0), warp_sums, all);
    if (e < a.experts) {
        place_of[e] = at.x + before, octet_of[e] = tiled ? -1 : at.y * 8 + before;
        if (rank == 0) {
            for (int i = 0, s = at.z; i < rows_n; i += 8 * kSetOctets, ++s)
                a.plan.sets[s] = {e, at.x + i, min(8 * kSetOctets, n - i), at.y + i / 8};
            for (int i = 0; i < (tiled ? tile_n : 0); ++i) a.plan.tile_sets[at.w + i] = {e, at.x + i * per, min(per, n - i * per), 0};
        }
    }
    if (e == 0 && rank == 0) a.plan.head[0] = all.z, a.plan.head[1] = all.w, a.plan.head[2] = all.x;
    __syncthreads();
    over_run([&](int64_t i, int id, bool live, unsigned same) {
        const int taken = live ? mine[id] : 0;
        __syncwarp();
        if (live) {
            const int k = taken + __popc(same & ((1u << lane) - 1));       // its number among this block's of the expert
            if (lane == __ffs(same) - 1) mine[id] = taken + __popc(same);
            const int p = place_of[id] + k;
            a.plan.place[i] = p;
            a.plan.column[p] = octet_of[id] < 0 ? -1 : octet_of[id] + k;
        } else if (i < last) {
            a.plan.place[i] = id < 0 ? -1 : -2;
        }
    });
    if (blocks > 1) cluster_sync();             // the counts are read to the end
}

__device__ __forceinline__ uint32_t pack2h(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Four scaled values as hi (and lo) pieces, in the order (0, 2, 1, 3) that taking nibbles and bytes apart by masks gives.
__device__ __forceinline__ void pieces_of(const float4 v, uint2 &hi, uint2 &lo)
{
    hi = make_uint2(pack2h(v.x, v.z), pack2h(v.y, v.w));
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&hi.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi.y));
    lo = make_uint2(pack2h(v.x - a.x, v.z - a.y), pack2h(v.y - b.x, v.w - b.y));
}

constexpr int kPackThreads = 256;

// Lays rows out as operands, WARPS warps a row: a token's row for each of its places (top_k > 0), or a place's own.
template <int WARPS>
__global__ void __launch_bounds__(kPackThreads) pack_kernel(const PackArgs a)
{
    constexpr int kThreads = 32 * WARPS;
    __shared__ uint32_t warp_max[kPackThreads / 32];
    let_next_start();
    wait_for_previous();
    const int tid = threadIdx.x % kThreads;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * (kPackThreads / kThreads) + threadIdx.x / kThreads;
    if (r >= (a.top_k ? a.tokens : a.plan.head[2])) return;         // (whole rows: all of a block's threads, or of a warp)
    const int64_t row = r * a.ld;
    // where blocks are few, one a place of the token's; a lane looks up one of up to 32 at once
    const int lane = threadIdx.x & 31;
    const int first = gridDim.y > 1 ? blockIdx.y : 0, places = gridDim.y > 1 ? first + 1 : a.top_k ? a.top_k : 1;
    int p = -1, column = 0;
    const auto look = [&](int j) {
        p = j >= places ? -1 : a.top_k ? a.plan.place[r * a.top_k + j] : static_cast<int>(r);
        column = p >= 0 ? a.plan.column[p] : 0;
    };
    look(first + lane);
    // short rows stay in registers: eight neighbouring values of every 256 (kThreads of them)
    constexpr int kHeld = WARPS == 1 ? 4 : 1;
    const bool hold = a.cols <= kHeld * kThreads * 8;
    float4 held[kHeld][2];
    uint32_t most = 0;          // magnitudes order as their bits do
    const auto look_at = [&](const float4 v) {
        most = max(max(most, max(__float_as_uint(v.x) & 0x7fffffffu, __float_as_uint(v.y) & 0x7fffffffu)),
                   max(__float_as_uint(v.z) & 0x7fffffffu, __float_as_uint(v.w) & 0x7fffffffu));
    };
    if (hold) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int k = (i * kThreads + tid) * 8 + 4 * q;
                held[i][q] = k < a.cols ? four(a.x, row, k, a.cols, a.type, a.vec) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) look_at(held[i][0]), look_at(held[i][1]);
    } else {
#pragma unroll 4
        for (int k = tid * 4; k < a.cols; k += kThreads * 4) look_at(four(a.x, row, k, a.cols, a.type, a.vec));
    }
    most = __reduce_max_sync(~0u, most);
    if constexpr (WARPS > 1) {
        if ((tid & 31) == 0) warp_max[tid >> 5] = most;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WARPS; ++w) most = max(most, warp_max[w]);
    }
    // 2^e puts it into [2^14, 2^15); rows of zeros, infinities and NaN stay as they are, and e stops where 2^-e is
    // no normal number any more
    const int ex = most >= 0x7f800000u || most == 0 ? 141 : max(static_cast<int>(most >> 23), 15);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 141 - ex) << 23);
    const float back = __uint_as_float(static_cast<uint32_t>(127 - 141 + ex) << 23);
    const int64_t unit = octet_unit_bytes(a.fmt, a.pieces);
    for (int j0 = first; j0 < places; j0 += 32) {
        if (j0 > first) look(j0 + lane);
        if (tid < 32 && p >= 0) a.scale[p] = back;
        const unsigned to_rows = __ballot_sync(~0u, p >= 0 && column >= 0), to_tiles = __ballot_sync(~0u, p >= 0 && column < 0);
        for (unsigned who = to_rows; who; who &= who - 1) {
            const int at_column = __shfl_sync(~0u, column, __ffs(who) - 1);
            // thread (unit, c, i) makes the 16 bytes that lane (column, c) of step i reads
            uint8_t *out = a.out + (at_column >> 3) * unit * a.units;
            const int col = at_column & 7;
            for (int q = tid; q < a.units * 32; q += kThreads) {
                const int u = q >> 5, c = (q >> 3) & 3, i = q & 7;
                const int k = u * kUnit;
                int k0, k1;
                if (a.fmt == kFmtQ4K) k0 = k + 64 * c + 4 * i, k1 = k0 + 32;                     // sub-blocks 2c and 2c + 1
                else if (a.fmt == kFmtQ80) k0 = k + 32 * i + 8 * c, k1 = k0 + 4;                 // block i
                else k0 = k + 128 * (i >> 2) + 64 * (i & 1) + 16 * ((i >> 1) & 1) + 4 * c, k1 = k0 + 32;    // sub-blocks t, t + 1
                float4 v0 = four(a.x, row, k0, a.cols, a.type, a.vec), v1 = four(a.x, row, k1, a.cols, a.type, a.vec);
                v0.x *= up, v0.y *= up, v0.z *= up, v0.w *= up;
                v1.x *= up, v1.y *= up, v1.z *= up, v1.w *= up;
                uint2 h0, l0, h1, l1;
                pieces_of(v0, h0, l0), pieces_of(v1, h1, l1);
                uint8_t *at = out + u * unit;
                const int slot = col * 4 + c;
                *reinterpret_cast<uint4 *>(at + i * 512 + slot * 16) = make_uint4(h0.x, h0.y, h1.x, h1.y);
                if (a.pieces == 2)
                    *reinterpret_cast<uint4 *>(at + kPieceBytes + i * 512 + slot * 16) = make_uint4(l0.x, l0.y, l1.x, l1.y);
                if (a.fmt == kFmtQ4K) {
                    // sums of the values as the pieces hold them, over the 8 threads of a sub-block; 2^-5 of them in two pieces
                    const auto held = [&](uint2 h, uint2 l) {
                        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&h.x));
                        const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&h.y));
                        float s = (x.x + x.y) + (y.x + y.y);
                        if (a.pieces == 2) {
                            const float2 z = __half22float2(*reinterpret_cast<const __half2 *>(&l.x));
                            const float2 w = __half22float2(*reinterpret_cast<const __half2 *>(&l.y));
                            s += (z.x + z.y) + (w.x + w.y);
                        }
                        return s;
                    };
                    float s0 = held(h0, l0), s1 = held(h1, l1);
    #pragma unroll
                    for (int d = 1; d < 8; d *= 2) s0 += __shfl_xor_sync(~0u, s0, d), s1 += __shfl_xor_sync(~0u, s1, d);
                    s0 *= 0.03125f, s1 *= 0.03125f;
                    if (i == 0) {
                        const uint32_t hi = pack2h(s0, s1);
                        const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                        *reinterpret_cast<uint2 *>(at + a.pieces * kPieceBytes + slot * 8) =
                            make_uint2(hi, pack2h(s0 - h.x, s1 - h.y));
                    }
                }
            }
        }
        if (!to_tiles) continue;
        // rows of tile sets, in the order in which their weights are taken apart: (0, 2, 1, 3) of every four
        const auto store = [&](int k, float4 v, float4 w) {
            v.x *= up, v.y *= up, v.z *= up, v.w *= up;
            w.x *= up, w.y *= up, w.z *= up, w.w *= up;
            uint2 h0, l0, h1, l1;
            pieces_of(v, h0, l0), pieces_of(w, h1, l1);
            for (unsigned who = to_tiles; who; who &= who - 1) {
                __half *to = a.tile_out + static_cast<int64_t>(__shfl_sync(~0u, p, __ffs(who) - 1)) * a.tile_cols + k;
                if (k < a.tile_cols) {
                    *reinterpret_cast<uint4 *>(to) = make_uint4(h0.x, h0.y, h1.x, h1.y);
                    if (a.pieces == 2) *reinterpret_cast<uint4 *>(to + a.tile_lo) = make_uint4(l0.x, l0.y, l1.x, l1.y);
                }
            }
        };
        if (hold) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) store((i * kThreads + tid) * 8, held[i][0], held[i][1]);
        } else {
            for (int k = tid * 8; k - tid * 8 < a.tile_cols; k += kThreads * 8) {
                const bool in = k < a.tile_cols;
                store(k, four(a.x, row, in ? k : 0, a.cols, a.type, a.vec), four(a.x, row, in ? k + 4 : 0, a.cols, a.type, a.vec));
            }
        }
    }
}

struct SumArgs {
    Plan plan;
    const float *parts;       // [place][N]
    const float *weights;
    int top_k, N, type;
    void *y;
    int64_t ldy;
};

constexpr int kSumThreads = 256;

// y[t] = sum over j, in order, of weights[t][j] * the part of assignment (t, j).
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const SumArgs a)
{
    let_next_start();
    wait_for_previous();
    const int64_t t = blockIdx.x;
    const int n = (blockIdx.y * kSumThreads + threadIdx.x) * 4;
    if (n >= a.N) return;
    const bool vec = a.N % 4 == 0;
    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int kAhead = 8;                   // parts on their way at once
    for (int j0 = 0; j0 < a.top_k; j0 += kAhead) {
        int p[kAhead];
        float w[kAhead], v[kAhead][4];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) p[i] = j0 + i < a.top_k ? a.plan.place[t * a.top_k + j0 + i] : -1;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            w[i] = p[i] >= 0 ? a.weights[t * a.top_k + j0 + i] : p[i] == -1 ? 0.0f : __int_as_float(0x7fc00000);
            const float *part = a.parts + static_cast<int64_t>(p[i]) * a.N + n;
            v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.0f;
            if (p[i] >= 0 && vec) {
                const float4 f = *reinterpret_cast<const float4 *>(part);
                v[i][0] = f.x, v[i][1] = f.y, v[i][2] = f.z, v[i][3] = f.w;
            } else if (p[i] >= 0) {
                for (int k = 0; k < 4; ++k) v[i][k] = n + k < a.N ? part[k] : 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] += w[i] * v[i][k];
    }
    for (int i = 0; i < 4 && n + i < a.N; ++i) store_float_as(a.y, t * a.ldy + n + i, a.type, y[i]);
}

// ---------------------------------------------------------------- the call

struct Layout {
    int64_t A, octets, sets, tile_sets;
    int pieces, w_pieces, tile_tokens;
    bool few;                 // few assignments: only h is used
    bool tiled;               // some expert may have enough tokens for the tile form
    int64_t head, place, column, set, tile_set, x_scale, h_scale, x, x_tile, h, h_ops, h_tile, parts, bytes;
};
int64_t tile_cols(int64_t cols) { return (cols + 127) / 128 * 128; }

int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

// Where a call's scratch lies.  The types decide how many pieces an operand has.
Layout layout_of(int64_t T, int top_k, int64_t E, int64_t K, int64_t F, int64_t N, int gate_fmt, int down_fmt, int x_type,
                 int y_type)
{
    Layout l{};
    l.A = T * top_k;
    l.pieces = x_type == QK_F32 || y_type == QK_F32 ? 2 : 1;
    l.w_pieces = x_type == QK_BF16 && y_type == QK_BF16 ? 1 : 2;
    l.tile_tokens = 128;
    // (an id may repeat within a token: such an expert goes by the few-token form, however many it has)
    l.few = l.A <= kMaxFew && K <= kMaxFewCols && F <= kMaxFewCols;
    if (l.few) {
        // groups of 16 values and their sum, whole runs of 256
        l.bytes = up256(l.A * ((F + 255) / 256 * 256) / 16 * 20 * 4);
        return l;
    }
    l.tiled = T >= kTileFrom;
    const int64_t used = std::min(l.A, E);
    // with the many-token form: experts of fewer than kTileFrom tokens, or sets a quarter as many again as those
    l.octets = l.tiled ? std::min(used + l.A / 8, 2 * E + (E / 4 + 1) * kSetOctets) : used + l.A / 8;
    l.sets = used + l.A / (8 * kSetOctets);
    l.tile_sets = l.tiled ? l.A / 64 + used : 0;
    int64_t at = 0;
    const auto take = [&](int64_t n) {
        const int64_t was = at;
        at += up256(n);
        return was;
    };
    const auto operands = [&](int fmt, int64_t cols) {
        return l.octets * ((cols + kUnit - 1) / kUnit) * octet_unit_bytes(fmt, l.pieces);
    };
    l.head = take(64), l.place = take(4 * l.A), l.column = take(4 * l.A);
    l.set = take(l.sets * sizeof(ExpertSet)), l.tile_set = take(l.tile_sets * sizeof(ExpertSet));
    const auto rows = [&](int64_t cols) { return l.tiled ? 2 * l.pieces * l.A * tile_cols(cols) : 0; };
    l.x_scale = take(4 * l.A), l.h_scale = take(4 * l.A);
    l.x = take(operands(gate_fmt, K)), l.x_tile = take(rows(K));
    l.h = take(4 * l.A * F), l.h_ops = take(operands(down_fmt, F)), l.h_tile = take(rows(F));
    l.parts = take(4 * l.A * N);
    l.bytes = at;
    return l;
}

bool multiple(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool type_ok(int t) { return t == QK_F32 || t == QK_F16 || t == QK_BF16; }
bool format_ok(int f) { return f == kFmtQ80 || f == kFmtQ4K || f == kFmtQ6K; }
int size_of(int t) { return t == QK_F32 ? 4 : 2; }

bool sizes_too_large(int64_t T, int top_k, int64_t E, int64_t K, int64_t F, int64_t N)
{
    return E > kMaxExperts || K > (1 << 24) || F > (1 << 24) || N > (1 << 24) || T > (1 << 28) / top_k;
}

// An expert tensor's rows of `cols` columns, `rows` of each expert (a qk_status).
int check_weights(const qk_expert_weights *w, int64_t E, int64_t rows, int64_t cols, Weights *out)
{
    if (!w || !w->w) return QK_ERR_NULL;
    if (!format_ok(w->format)) return QK_ERR_TYPE;
    const int64_t per = w->expert_rows == 0 ? rows : w->expert_rows;
    if (w->row_offset < 0 || per < rows) return QK_ERR_BAD_DIM;
    if (strict_blocks_reject(w->format, cols)) return QK_ERR_BAD_DIM;
    const int64_t rb = row_bytes_of(w->format, cols);
    if (per > INT32_MAX / E || w->row_offset > INT64_MAX / rb - E * per) return QK_ERR_TOO_LARGE;
    if (!multiple(w->w, w->format == kFmtQ4K ? 16 : 2)) return QK_ERR_ALIGN;
    *out = {static_cast<const uint8_t *>(w->w) + w->row_offset * rb, per, rb};
    return QK_OK;
}

template <class F>
F *by_format(int fmt, F *q4k, F *q80, F *q6k)
{
    return fmt == kFmtQ4K ? q4k : fmt == kFmtQ80 ? q80 : q6k;
}

}  // namespace
}  // namespace qk

using namespace qk;

extern "C" {

// Test hook, not part of the public header: the first thread blocks of later
// many-token launches never load chunk number `chunk` of the tokens (-1: off),
// so that a bounded wait runs out and the launch records QK_ERR_TIMEOUT.
int qk_debug_moe_skip_chunk(int chunk) { return g_skip_chunk.exchange(chunk); }

size_t qk_moe_ffn_workspace_bytes(int64_t T, int top_k, int64_t n_experts, int64_t K, int64_t F, int64_t N)
{
    if (T <= 0 || top_k <= 0 || n_experts <= 0 || K <= 0 || F <= 0 || N <= 0) return 0;
    if (sizes_too_large(T, top_k, n_experts, K, F, N)) return 0;
    const auto bytes = [&](int64_t t) { return layout_of(t, top_k, n_experts, K, F, N, kFmtQ4K, kFmtQ4K, QK_F32, QK_F32).bytes; };
    // with more ids a token than experts the most tokens that go without the many-token form can need more than a few more do
    return static_cast<size_t>(std::max(bytes(T), bytes(std::min<int64_t>(T, kTileFrom - 1))));
}

int qk_moe_ffn(const qk_expert_weights *gate, const qk_expert_weights *up, const qk_expert_weights *down, int64_t n_experts,
               int64_t K, int64_t F, int64_t N, const void *x, int64_t ldx, int x_type, int64_t T, const int32_t *ids,
               const float *weights, int top_k, void *y, int64_t ldy, int y_type, void *workspace, size_t workspace_bytes,
               qk_stream_t stream)
{
    if (!gate || !up || !down) return QK_ERR_NULL;
    if (!type_ok(x_type) || !type_ok(y_type) || gate->format != up->format) return QK_ERR_TYPE;
    if (n_experts <= 0 || K <= 0 || F <= 0 || N <= 0 || T < 0 || top_k <= 0) return QK_ERR_BAD_DIM;
    if (ldx == 0) ldx = K;
    if (ldy == 0) ldy = N;
    if (ldx < K || ldy < N) return QK_ERR_BAD_DIM;
    if (sizes_too_large(T, top_k, n_experts, K, F, N)) return QK_ERR_TOO_LARGE;
    Weights wg, wu, wd;
    int st = check_weights(gate, n_experts, F, K, &wg);
    if (st == QK_OK) st = check_weights(up, n_experts, F, K, &wu);
    if (st == QK_OK) st = check_weights(down, n_experts, N, F, &wd);
    if (st != QK_OK) return st;
    // the kernels count items: a set of tokens, and 32 rows of gate and up, or of down
    if ((static_cast<int64_t>(T) * top_k / 16 + n_experts) * ((std::max(2 * F, N) + 31) / 32) > INT32_MAX) return QK_ERR_TOO_LARGE;
    if (T == 0) return QK_OK;
    if (!x || !ids || !weights || !y) return QK_ERR_NULL;
    if (!multiple(x, size_of(x_type)) || !multiple(y, size_of(y_type)) || !multiple(ids, 4) || !multiple(weights, 4))
        return QK_ERR_ALIGN;
    const Layout l = layout_of(T, top_k, n_experts, K, F, N, gate->format, down->format, x_type, y_type);
    if (!workspace || !multiple(workspace, 256) || workspace_bytes < static_cast<size_t>(l.bytes)) return QK_ERR_WORKSPACE;
    int sms = 0, smem = 0;
    int *err = library_error_word();
    if (!err || !device_limits(&sms, &smem)) return QK_ERR_CUDA;
    char *ws = static_cast<char *>(workspace);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);

    if (l.few) {
        FewArgs f{};
        f.ids = ids, f.experts = static_cast<int>(n_experts), f.top_k = top_k, f.err = err;
        f.a = wg, f.b = wu, f.cols = static_cast<int>(K), f.rows = static_cast<int>(F);
        f.x = x, f.ldx = ldx, f.x_type = x_type, f.vec = multiple(x, 4 * size_of(x_type)) && ldx % 4 == 0;
        f.h = reinterpret_cast<float *>(ws + l.h);
        f.weights = weights, f.y = y, f.ldy = ldy, f.y_type = y_type;
        cudaError_t e = by_format(gate->format, few_gate_q4k, few_gate_q80, few_gate_q6k)(f, l.A, down->format, library_programmatic(), s);
        f.a = wd, f.cols = static_cast<int>(F), f.rows = static_cast<int>(N);
        if (e == cudaSuccess) e = by_format(down->format, few_down_q4k, few_down_q80, few_down_q6k)(f, T, s);
        return e == cudaSuccess ? QK_OK : QK_ERR_CUDA;
    }

    PlanArgs pa{};
    pa.ids = ids, pa.n = static_cast<int>(l.A), pa.experts = static_cast<int>(n_experts), pa.err = err;
    // 8 thread blocks where one would go over its ids more than once (4096 ids: 15 us in one and 12 in 8; 32768: 82 and 16)
    constexpr int kWarps = kPlanThreads / 32;
    const int plan_blocks = l.A > 32 * kWarps ? 8 : 1;
    pa.per_warp = static_cast<int>((l.A + 32LL * kWarps * plan_blocks - 1) / (32LL * kWarps * plan_blocks) * 32);
    pa.plan = {reinterpret_cast<int *>(ws + l.head), reinterpret_cast<int *>(ws + l.place), reinterpret_cast<int *>(ws + l.column),
               reinterpret_cast<ExpertSet *>(ws + l.set), reinterpret_cast<ExpertSet *>(ws + l.tile_set)};
    pa.tile_from = l.tiled ? kTileFrom : INT32_MAX, pa.tile_tokens = l.tile_tokens;
    const size_t counts = sizeof(int) * kWarps * pa.experts;
    cudaError_t e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(sizeof(int) * kWarps * kMaxExperts));
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(plan_blocks), cfg.blockDim = dim3(kPlanThreads), cfg.dynamicSmemBytes = counts, cfg.stream = s;
        cudaLaunchAttribute at[2]{};
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = plan_blocks, at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at, cfg.numAttrs = library_programmatic() ? 2 : 1;
        e = cudaLaunchKernelEx(&cfg, plan_kernel, pa);
    }
    if (e != cudaSuccess) return QK_ERR_CUDA;

    const auto pack = [&](const void *rows, int64_t ld, int type, int per_row, int64_t cols, int fmt, int64_t to, int64_t tile_to, int64_t scale) {
        PackArgs k{};
        k.tile_out = reinterpret_cast<__half *>(ws + tile_to), k.tile_cols = static_cast<int>(tile_cols(cols)), k.tile_lo = l.A * k.tile_cols;
        k.plan = pa.plan, k.x = rows, k.ld = ld, k.type = type, k.top_k = per_row;
        k.cols = static_cast<int>(cols), k.units = static_cast<int>((cols + kUnit - 1) / kUnit);
        k.pieces = l.pieces, k.fmt = fmt;
        k.out = reinterpret_cast<uint8_t *>(ws + to), k.scale = reinterpret_cast<float *>(ws + scale);
        k.vec = multiple(rows, 4 * size_of(type)) && ld % 4 == 0, k.tokens = T;
        // a thread block a row where rows are few, else a warp
        const int64_t n = per_row ? T : l.A;
        const bool wide = n <= 4LL * sms;
        return wide ? launch_chained(pack_kernel<kPackThreads / 32>, dim3(static_cast<unsigned>(n), per_row && n * per_row <= 4LL * sms ? per_row : 1),
                                     kPackThreads, 0, s, true, k)
                    : launch_chained(pack_kernel<1>, dim3(static_cast<unsigned>((n + kPackThreads / 32 - 1) / (kPackThreads / 32))),
                                     kPackThreads, 0, s, true, k);
    };
    const auto products = [&](const Weights &a, const Weights &b, int fmt, int64_t cols, int64_t rows, bool paired,
                              int64_t ops, int64_t tile_ops, int64_t scale, int64_t to) {
        if (l.tiled) {
            const int64_t wide = tile_cols(cols);
            const TileOperands o = {ws + tile_ops, ws + tile_ops + 2 * l.A * wide, l.A, wide};
            TileArgs t{};
            t.plan = pa.plan, t.a = a, t.b = b, t.cols = static_cast<int>(cols), t.chunks = static_cast<int>(wide / (l.w_pieces == 1 ? 128 : 64));
            t.pieces = l.pieces, t.w_pieces = l.w_pieces, t.rows = static_cast<int>(rows);
            t.tiles = static_cast<int>(paired ? (rows + 63) / 64 : (rows + 127) / 128);
            t.scale = reinterpret_cast<const float *>(ws + scale), t.out = reinterpret_cast<float *>(ws + to);
            t.skip_chunk = g_skip_chunk.load(), t.wait_ns = library_wait_limit_ns(), t.err = err;
            const cudaError_t e = by_format(fmt, tile_launch_q4k, tile_launch_q80, tile_launch_q6k)(o, t, paired, sms, s);
            if (e != cudaSuccess) return e;
        }
        RowsArgs r{};
        r.plan = pa.plan, r.a = a, r.b = b;
        r.cols = static_cast<int>(cols), r.units = static_cast<int>((cols + kUnit - 1) / kUnit), r.pieces = l.pieces;
        r.rows = static_cast<int>(rows), r.tiles = static_cast<int>(paired ? (rows + 7) / 8 : (rows + 15) / 16);
        r.sms = sms, r.wait_ns = library_wait_limit_ns(), r.err = err;
        r.x = reinterpret_cast<const uint8_t *>(ws + ops), r.scale = reinterpret_cast<const float *>(ws + scale);
        r.out = reinterpret_cast<float *>(ws + to);
        return by_format(fmt, rows_launch_q4k, rows_launch_q80, rows_launch_q6k)(r, paired, sms, s);
    };
    e = pack(x, ldx, x_type, top_k, K, gate->format, l.x, l.x_tile, l.x_scale);
    if (e == cudaSuccess) e = products(wg, wu, gate->format, K, F, true, l.x, l.x_tile, l.x_scale, l.h);
    if (e == cudaSuccess) e = pack(ws + l.h, F, QK_F32, 0, F, down->format, l.h_ops, l.h_tile, l.h_scale);
    if (e == cudaSuccess) e = products(wd, wd, down->format, F, N, false, l.h_ops, l.h_tile, l.h_scale, l.parts);
    if (e != cudaSuccess) return QK_ERR_CUDA;
    SumArgs u{};
    u.plan = pa.plan, u.parts = reinterpret_cast<const float *>(ws + l.parts), u.weights = weights;
    u.top_k = top_k, u.N = static_cast<int>(N), u.type = y_type, u.y = y, u.ldy = ldy;
    e = launch_chained(sum_kernel, dim3(static_cast<unsigned>(T), static_cast<unsigned>((N + 4 * kSumThreads - 1) / (4 * kSumThreads))),
                       kSumThreads, 0, s, true, u);
    return e == cudaSuccess ? QK_OK : QK_ERR_CUDA;
}

}  // extern "C"
