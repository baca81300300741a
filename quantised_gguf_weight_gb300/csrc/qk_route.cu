// qk_route.cu -- routing to experts: scores of a token's logits, the choice of
// its top_k experts and their weights.
//
// A warp takes a token; lane l has the experts [l V, (l + 1) V).  A choice is a
// maximum over a lane's keys, one redux over the warp and the lowest lane that
// has it, so ties go to the lowest index.  A key is the value's bits, mapped so
// that unsigned order is the values' order.
//
// Where a score is only a rising function of its logit (no bias, and groups
// that count as their best expert), the logits themselves are compared and the
// order is exact.  Else scores are compared, first in 32 bits with a bound on
// their error; a token in which that leaves two neighbours of the order, or a
// group at the edge, undecided is done again in 64 bits (about 1 in 2000 tokens
// of 256 experts in groups; a launch that has one takes 14 us longer).  So the
// choice is that of the formulas, not of a rounding.
//
// A weight is off by at most 19 x 2^-24 of itself: softmax over all experts, two exponentials 2^-23 each, their arguments'
// rests 2^-24 each, ten additions, the division and the scale; sigmoid over its sum, six for each score, five additions, the
// division and the scale.
//
// Measured, calls one after another in a graph: one token 2.9 us, which is a
// launch; 512 tokens of 256 experts in groups 6.6, or 20.7 where a token is done
// again; 16384 tokens of 128 experts in bf16 11.4 us, bound by instructions (0.66
// a cycle and scheduler), 4.3 MB read.
#include <cmath>

#include "qk_kv4.cuh"
#include "qk_moe.cuh"

namespace qk {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxExperts = 1024;

struct RouteArgs {
    const void *logits;
    int64_t ld, T;
    int type, E, top_k, sigmoid, groups, top_groups, group_top, renorm, by_logits;
    const float *bias;
    float scale;
    int32_t *ids;
    float *weights;
    bool vec;
};

__device__ __forceinline__ uint32_t key_of(float v)
{
    const uint32_t b = __float_as_uint(v + 0.0f);        // one zero
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(double v)
{
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
    return b >> 63 ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
__device__ __forceinline__ double value_of(uint64_t k)
{
    return __longlong_as_double(static_cast<long long>(k >> 63 ? k & 0x7fffffffffffffffull : ~k));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(~0u, k); }
__device__ __forceinline__ uint64_t warp_max(uint64_t k)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const uint64_t o = __shfl_xor_sync(~0u, k, d);
        k = o > k ? o : k;
    }
    return k;
}
template <class R>
__device__ __forceinline__ R warp_sum(R v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    return v;
}
__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }
__device__ __forceinline__ float most_of(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double most_of(double a, double b) { return a > b ? a : b; }
__device__ __forceinline__ float least_of(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double least_of(double a, double b) { return a > b ? b : a; }
// e^(a - b) for a <= b: the difference with what its rounding leaves (an argument of 80 rounded by itself is 4e-6 of the result)
__device__ __forceinline__ float exp_less(float a, float b)
{
    const float d = a - b, back = d - a, rest = (a - (d - back)) - (b + back), v = expf(d);
    return d > -INFINITY ? fmaf(v, rest, v) : 0.0f;
}
// By halves: an addition's error meets each term V's logarithm times, not V times.
template <class R, int V>
__device__ __forceinline__ R sum_of(const R (&v)[V])
{
    R s[V];
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = v[i];
#pragma unroll
    for (int n = V / 2; n > 0; n /= 2)
#pragma unroll
        for (int i = 0; i < n; ++i) s[i] += s[i + n];
    return s[0];
}

template <class R>
struct KeyOf;
template <>
struct KeyOf<float> { using type = uint32_t; };
template <>
struct KeyOf<double> { using type = uint64_t; };

// Chooses top_k experts: lane j gets the j-th one's index and logit.  False where 32 bits leave the order open.
template <class R, int V>
__device__ __forceinline__ bool choose(const RouteArgs &a, const float (&z)[V], float zmax, R *shared, int lane, int &index,
                                       float &logit)
{
    using Key = typename KeyOf<R>::type;
    constexpr bool kWide = sizeof(R) == 8;
    const bool by_logits = a.by_logits;
    // A score's error in 32 bits, of itself: an exponential's 2^-23, the sum 1 + e^-z and the division 2^-24 each; softmax:
    // the argument's 2^-18 (differences of 64 to 128), and ten additions.  Scores below the normal numbers have few bits or
    // none.  And the error of its sum with the bias, twice the rounding's 2^-24.
    const R of_score = a.sigmoid ? R(4e-7) : R(5e-6), of_sum = R(1.2e-7), least = R(1e-37);
    R c[V], err[V];
    R total = 0;
    if (!by_logits && !a.sigmoid) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const bool in = lane * V + v < a.E;
            c[v] = in && z[v] > -INFINITY ? exp_of(R(z[v]) - R(zmax)) : R(0);
        }
        total = warp_sum(sum_of(c));
    }
    const int each = a.E / a.groups;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane * V + v;
        err[v] = 0;
        if (by_logits) {
            c[v] = R(z[v]);
        } else {
            c[v] = a.sigmoid ? R(1) / (R(1) + exp_of(-R(z[v]))) : (total > R(0) ? c[v] / total : R(0));
            if (!kWide) err[v] = c[v] * of_score + least;
            if (a.bias && e < a.E) c[v] += R(__ldg(a.bias + e));
            if (!kWide) err[v] = isinf(c[v]) ? R(0) : err[v] + fabsf(static_cast<float>(c[v])) * of_sum;
        }
    }
    bool open = false;
    unsigned kept = ~0u;
    if (a.groups > 1) {
        // A group's value lies between the sum of its best lower ends and that of its best upper ends, whatever is added up
        // in it (biases may cancel); without errors both are the value.
        const bool bounds = !kWide && !by_logits;
        float2 *ends = reinterpret_cast<float2 *>(shared);       // (32 bits: as many bytes as 64 bits have)
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (lane * V + v < a.E) {
                if (bounds) ends[lane * V + v] = make_float2(c[v] + err[v], c[v] - err[v]);
                else shared[lane * V + v] = c[v];
            }
        __syncwarp();
        R first = -INFINITY, second = -INFINITY, low_first = -INFINITY, low_second = -INFINITY;
        const auto take = [](R &best, R &next, R s) {
            next = most_of(next, least_of(best, s));
            best = most_of(best, s);
        };
        // (lanes start apart: fewer bank conflicts)
        int at = lane % each;
        if (lane < a.groups && bounds) {
#pragma unroll 2
            for (int i = 0; i < each; ++i, at = at + 1 == each ? 0 : at + 1) {
                const float2 s = ends[lane * each + at];
                take(first, second, s.x), take(low_first, low_second, s.y);
            }
        } else if (lane < a.groups) {
#pragma unroll 2
            for (int i = 0; i < each; ++i, at = at + 1 == each ? 0 : at + 1) take(first, second, shared[lane * each + at]);
        }
        __syncwarp();
        const R sum = a.group_top == 2 ? first + second : first;
        const Key mine = lane < a.groups ? key_of(sum) : Key(0);
        int better = 0;
        for (int o = 0; o < a.groups; ++o) {
            const Key other = __shfl_sync(~0u, mine, o);
            better += other > mine || (other == mine && o < lane);
        }
        const bool keep = lane < a.groups && better < a.top_groups;
        kept = __ballot_sync(~0u, keep);
        if (bounds) {
            // the worst that is kept and the best that is not, whose sums are rounded themselves
            const R low = a.group_top == 2 ? low_first + low_second : low_first;
            const R worst = value_of(static_cast<Key>(~warp_max(keep ? static_cast<Key>(~key_of(low)) : Key(0))));
            const R best = value_of(warp_max(!keep && lane < a.groups ? mine : Key(0)));
            open = best > R(-INFINITY) && !(worst - best > of_sum * (fabsf(static_cast<float>(worst)) + fabsf(static_cast<float>(best))));
        }
    }
    Key key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane * V + v;
        key[v] = e < a.E && (a.groups == 1 || (kept >> (e / each)) & 1u) ? key_of(c[v]) : Key(0);
    }
    if (by_logits) {
        // the key is the logit
        if (!kWide && a.type != QK_F32) {
            // 16-bit logits have 19 bits of key at most: the index goes with them, lower ones first
            uint32_t both[V];
#pragma unroll
            for (int v = 0; v < V; ++v) both[v] = key[v] ? (static_cast<uint32_t>(key[v]) >> 13 << 11) + (kMaxExperts - (lane * V + v)) : 0u;
            for (int j = 0; j < a.top_k; ++j) {
                uint32_t best = both[0];
#pragma unroll
                for (int v = 1; v < V; ++v) best = max(best, both[v]);
                const uint32_t top = __reduce_max_sync(~0u, best);
                if (lane == j) {
                    const uint32_t k = top >> 11 << 13;
                    index = kMaxExperts - (top & 2047u), logit = __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~(k | 0x1fffu));
                }
#pragma unroll
                for (int v = 0; v < V; ++v) both[v] = both[v] == top ? 0u : both[v];
            }
            return true;
        }
        for (int j = 0; j < a.top_k; ++j) {
            Key best = key[0];
#pragma unroll
            for (int v = 1; v < V; ++v) best = key[v] > best ? key[v] : best;
            const Key top = warp_max(best);
            const int winner = __ffs(__ballot_sync(~0u, best == top)) - 1;
            int at = V - 1;
#pragma unroll
            for (int v = V - 2; v >= 0; --v) at = key[v] == top ? v : at;
            const int e = __shfl_sync(~0u, lane * V + at, winner);
            if (lane == j) index = e, logit = static_cast<float>(value_of(top));
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (lane * V + v == e) key[v] = 0;
        }
        return true;
    }
    R last_c = 0, last_err = 0;
    float last_z = 0, last_b = 0;
    for (int j = 0; j < a.top_k; ++j) {
        Key best = 0;
        int at = 0;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (key[v] > best) best = key[v], at = v;
        const Key top = warp_max(best);
        const int winner = __ffs(__ballot_sync(~0u, best == top)) - 1;
        float zw = 0;
        R ew = 0;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v == at) {
                zw = z[v], ew = err[v];
                if (lane == winner) key[v] = 0;
            }
        const int e = __shfl_sync(~0u, lane * V + at, winner);
        zw = __shfl_sync(~0u, zw, winner);
        if (lane == j) index = e, logit = zw;
        if (!kWide) {
            ew = __shfl_sync(~0u, ew, winner);
            const R cw = value_of(top);
            if (j > 0 && !(last_c - cw > last_err + ew)) {
                // the same logit and bias are a tie whatever the rounding
                const float bw = a.bias ? __ldg(a.bias + e) : 0.0f;
                if (!a.bias) last_b = 0.0f;
                open |= zw != last_z || bw != last_b;
            }
            last_c = cw, last_err = ew, last_z = zw;
            if (a.bias) last_b = __ldg(a.bias + e);
        }
    }
    if (!kWide) {
        // every one that is left has to be apart from the last, not only the next: its error may be larger
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (key[v] && !(last_c - c[v] > last_err + err[v]))
                open |= z[v] != last_z || (a.bias && __ldg(a.bias + lane * V + v) != last_b);
        open = __any_sync(~0u, open);
    }
    return !open;
}

template <int V>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const RouteArgs a)
{
    extern __shared__ double scratch[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    moe::let_next_start();
    moe::wait_for_previous();
    if (t >= a.T) return;
    double *shared = scratch + (a.groups > 1 ? warp * a.E : 0);
    float z[V];
    const int64_t row = t * a.ld;
    if (V >= 4 && a.vec) {
#pragma unroll
        for (int v = 0; v + 3 < V; v += 4) {
            const int64_t i = row + lane * V + v;
            if (a.type == QK_F32) {
                const float4 f = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.logits) + i);
                z[v] = f.x, z[v + 1] = f.y, z[v + 2] = f.z, z[v + 3] = f.w;
            } else {
                const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.logits) + i);
                const uint32_t u[2] = {w.x, w.y};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 f = a.type == QK_F16
                                         ? __half22float2(*reinterpret_cast<const __half2 *>(&u[k]))
                                         : make_float2(__uint_as_float(u[k] << 16), __uint_as_float(u[k] & 0xffff0000u));
                    z[v + 2 * k] = f.x, z[v + 2 * k + 1] = f.y;
                }
            }
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = lane * V + v;
            z[v] = e < a.E ? load_as_float(a.logits, row + e, a.type) : -INFINITY;
        }
    }
    bool bad = false;
    float zmax = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        bad |= isnan(z[v]) || (!a.sigmoid && z[v] == INFINITY);
        if (a.bias && lane * V + v < a.E) bad |= isnan(__ldg(a.bias + lane * V + v));
        zmax = fmaxf(zmax, z[v]);
    }
    bad = __any_sync(~0u, bad);
    zmax = value_of(warp_max(key_of(zmax)));
    int index = lane;
    float w = __int_as_float(0x7fc00000);
    if (!bad) {
        float logit = 0.0f;
        if (!choose<float, V>(a, z, zmax, reinterpret_cast<float *>(shared), lane, index, logit))
            choose<double, V>(a, z, zmax, shared, lane, index, logit);
        const bool mine = lane < a.top_k;
        // weights from the chosen logits: divided by their sum they need no other, and cannot all underflow
        const float most = value_of(warp_max(key_of(mine ? logit : -INFINITY)));
        if (a.sigmoid) {
            // below zero as e^z / (1 + e^z), which divided by their sum may all be times e^-most: none is lost that is left in it
            w = logit < 0.0f ? exp_less(logit, a.renorm ? fminf(most, 0.0f) : 0.0f) / (1.0f + expf(logit)) : 1.0f / (1.0f + expf(-logit));
        } else if (a.renorm) {
            w = exp_less(logit, most);
        } else {
            float s[V];
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] = exp_less(z[v], zmax);
            w = exp_less(logit, zmax) / warp_sum(sum_of(s));
        }
        if (!mine || !(logit > -INFINITY)) w = 0.0f;
        if (a.renorm) {
            const float s = warp_sum(w);
            w = s > 0.0f ? w / s : 0.0f;
        }
        w *= a.scale;
    }
    if (lane < a.top_k) {
        a.ids[t * a.top_k + lane] = index;
        a.weights[t * a.top_k + lane] = w;
    }
}

bool multiple(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace
}  // namespace qk

using namespace qk;

extern "C" int qk_moe_route(const void *logits, int64_t ld, int type, int64_t T, int n_experts, int top_k, int score,
                            const float *bias, int n_groups, int top_groups, int group_top, int renorm, float scale,
                            int32_t *ids, float *weights, qk_stream_t stream)
{
    if (type != QK_F32 && type != QK_F16 && type != QK_BF16) return QK_ERR_TYPE;
    if (score != QK_SOFTMAX && score != QK_SIGMOID) return QK_ERR_TYPE;
    if (T < 0 || n_experts <= 0 || top_k <= 0 || n_groups <= 0 || n_experts % n_groups || top_groups <= 0 ||
        top_groups > n_groups || group_top < 1 || group_top > 2 || !std::isfinite(scale))
        return QK_ERR_BAD_DIM;
    if (group_top > n_experts / n_groups || top_k > static_cast<int64_t>(top_groups) * (n_experts / n_groups))
        return QK_ERR_BAD_DIM;
    if (ld == 0) ld = n_experts;
    if (ld < n_experts) return QK_ERR_BAD_DIM;
    if (n_experts > kMaxExperts || top_k > 32 || n_groups > 32 || T > INT32_MAX) return QK_ERR_TOO_LARGE;
    if (T == 0) return QK_OK;
    if (!logits || !ids || !weights) return QK_ERR_NULL;
    const int size = type == QK_F32 ? 4 : 2;
    if (!multiple(logits, size) || !multiple(bias, 4) || !multiple(ids, 4) || !multiple(weights, 4)) return QK_ERR_ALIGN;
    RouteArgs a{};
    a.logits = logits, a.ld = ld, a.T = T, a.type = type, a.E = n_experts, a.top_k = top_k;
    a.sigmoid = score == QK_SIGMOID, a.groups = top_groups == n_groups ? 1 : n_groups, a.top_groups = top_groups;
    a.group_top = group_top, a.renorm = renorm != 0, a.bias = bias, a.scale = scale, a.ids = ids, a.weights = weights;
    a.by_logits = !bias && (a.groups == 1 || group_top == 1);
    int V = 1;
    while (32 * V < n_experts) V *= 2;
    a.vec = n_experts == 32 * V && ld % 4 == 0 && multiple(logits, 4 * size);
    const auto kern = V == 1 ? route_kernel<1> : V == 2 ? route_kernel<2> : V == 4 ? route_kernel<4>
                    : V == 8 ? route_kernel<8> : V == 16 ? route_kernel<16> : route_kernel<32>;
    const size_t smem = a.groups > 1 ? sizeof(double) * kWarps * n_experts : 0;
    const cudaError_t e = moe::launch_chained(kern, dim3(static_cast<unsigned>((T + kWarps - 1) / kWarps)), kWarps * 32, smem,
                                              reinterpret_cast<cudaStream_t>(stream), library_programmatic(), a);
    return e == cudaSuccess ? QK_OK : QK_ERR_CUDA;
}
