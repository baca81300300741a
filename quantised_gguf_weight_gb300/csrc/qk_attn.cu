// qk_attn.cu -- attention over the 4-bit paged cache (qk_attn_q4).
//
// First form: one block of four warps per query row and head; each warp takes
// every fourth key, a lane holds one channel of each scale group, and a
// running maximum and sum carry the softmax.
#include <cmath>

#include "qk_device.cuh"
#include "qk_internal.h"
#include "qk_kv4.cuh"

namespace qk {
namespace {

constexpr int kMaxGroups = 8;

struct AttnArgs {
    const uint8_t *pages;
    int64_t n_pages;
    int n_kv, D, page_tokens, n_q, rep;
    const void *q;
    int64_t ldq;
    int q_type;
    const int32_t *page_table;
    int64_t ld_pages, max_pages;
    const int32_t *lens, *q_start;
    int64_t B, T, max_q, window;
    float scale;
    void *out;
    int64_t ldo;
    int out_type;
    int *err;
};

__global__ void __launch_bounds__(128) attn_rows_kernel(const AttnArgs a)
{
    __shared__ float part[4][32 * kMaxGroups + 2];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t b = blockIdx.x / a.max_q, i = blockIdx.x - b * a.max_q;
    const int h = blockIdx.y, hk = h / a.rep, G = a.D / 32;
    int64_t r0 = b * a.max_q, r1 = r0 + a.max_q;
    if (a.q_start) r0 = a.q_start[b], r1 = a.q_start[b + 1];
    const int64_t L = a.lens[b];
    bool bad = L < 0 || L > a.max_pages * a.page_tokens;
    if (r0 < 0 || r1 > a.T || r1 < r0 || r1 - r0 > a.max_q) {
        bad = true;
        r0 = r0 < 0 ? 0 : r0;
        r1 = r1 > a.T ? a.T : r1;
    }
    if (bad && threadIdx.x == 0) record_error(a.err, kErrBadIndex);
    // a sequence whose row range is out of order may name more rows than blocks: each block takes a stride of them
    for (int64_t row = r0 + i; row < r1; row += a.max_q) {
        const int64_t pos = L - (r1 - row);
        float q[kMaxGroups], o[kMaxGroups];
#pragma unroll
        for (int g = 0; g < kMaxGroups; ++g) {
            o[g] = 0.0f;
            q[g] = g < G ? load_as_float(a.q, row * a.ldq + static_cast<int64_t>(h) * a.D + 32 * g + lane, a.q_type) *
                               a.scale
                         : 0.0f;
        }
        float m = -3.0e38f, l = 0.0f;
        int64_t j0 = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
        const int64_t j1 = bad ? 0 : pos + 1;
        bool poison = bad;
        for (int64_t j = j0 + warp; j < j1; j += 4) {
            const int32_t page = a.page_table[b * a.ld_pages + j / a.page_tokens];
            if (page < 0 || page >= a.n_pages) {
                if (lane == 0) record_error(a.err, kErrBadIndex);
                poison = true;
                continue;
            }
            const int off = static_cast<int>(j % a.page_tokens), t = off % kBlockTokens;
            const uint8_t *block = a.pages + ((static_cast<int64_t>(page) * a.n_kv + hk) *
                                                  (a.page_tokens / kBlockTokens) + off / kBlockTokens) *
                                                 static_cast<int64_t>(18 * a.D);
            float s = 0.0f, v[kMaxGroups];
#pragma unroll
            for (int g = 0; g < kMaxGroups; ++g) {
                v[g] = 0.0f;
                if (g < G) {
                    const Kv4Place pk = kv4_key_place(a.D, t, 32 * g + lane);
                    const Kv4Place pv = kv4_value_place(a.D, t, 32 * g + lane);
                    const float dk = __half2float(*reinterpret_cast<const __half *>(block + kv4_key_scale(a.D, t, g)));
                    const float dv = __half2float(*reinterpret_cast<const __half *>(block + kv4_value_scale(a.D, t, g)));
                    const uint32_t nk = *reinterpret_cast<const uint32_t *>(block + pk.byte) >> (4 * pk.nibble) & 15u;
                    const uint32_t nv = *reinterpret_cast<const uint32_t *>(block + pv.byte) >> (4 * pv.nibble) & 15u;
                    s = fmaf(q[g], dk * (static_cast<float>(nk) - 8.0f), s);
                    v[g] = dv * (static_cast<float>(nv) - 8.0f);
                }
            }
#pragma unroll
            for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
            const float m2 = fmaxf(m, s), f = expf(m - m2), p = expf(s - m2);
            m = m2;
            l = l * f + p;
#pragma unroll
            for (int g = 0; g < kMaxGroups; ++g) o[g] = fmaf(p, v[g], o[g] * f);
        }
        if (poison) l = __int_as_float(0x7FC00000);
#pragma unroll
        for (int g = 0; g < kMaxGroups; ++g) part[warp][32 * g + lane] = o[g];
        if (lane == 0) part[warp][32 * kMaxGroups] = m, part[warp][32 * kMaxGroups + 1] = l;
        __syncthreads();
        float mx = -3.0e38f, sum = 0.0f;
        for (int w = 0; w < 4; ++w) mx = fmaxf(mx, part[w][32 * kMaxGroups]);
        for (int w = 0; w < 4; ++w) sum += part[w][32 * kMaxGroups + 1] * expf(part[w][32 * kMaxGroups] - mx);
        for (int ch = threadIdx.x; ch < a.D; ch += 128) {
            float v = 0.0f;
            for (int w = 0; w < 4; ++w) v += part[w][ch] * expf(part[w][32 * kMaxGroups] - mx);
            store_float_as(a.out, row * a.ldo + static_cast<int64_t>(h) * a.D + ch, a.out_type,
                           sum == 0.0f ? 0.0f : v / sum);
        }
        __syncthreads();
    }
}

bool multiple(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool type_ok(int t) { return t == QK_F32 || t == QK_F16 || t == QK_BF16; }

}  // namespace
}  // namespace qk

using namespace qk;

extern "C" {

size_t qk_attn_q4_workspace_bytes(int64_t B, int n_q_heads, int n_kv_heads, int head_dim, int64_t max_q,
                                  int64_t max_len)
{
    (void)B, (void)n_q_heads, (void)n_kv_heads, (void)head_dim, (void)max_q, (void)max_len;
    return 0;
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
    if (n_q_heads > 65535 || B > INT32_MAX / max_q || T > INT32_MAX || max_pages > INT32_MAX / cache->page_tokens)
        return QK_ERR_TOO_LARGE;
    AttnArgs a{};
    a.pages = static_cast<const uint8_t *>(cache->pages), a.n_pages = cache->n_pages;
    a.n_kv = n_kv, a.D = D, a.page_tokens = cache->page_tokens, a.n_q = n_q_heads, a.rep = n_q_heads / n_kv;
    a.q = q, a.ldq = ldq, a.q_type = q_type;
    a.page_table = page_table, a.ld_pages = ld_pages, a.max_pages = max_pages;
    a.lens = lens, a.q_start = q_start, a.B = B, a.T = T, a.max_q = max_q, a.window = window, a.scale = scale;
    a.out = out, a.ldo = ldo, a.out_type = out_type;
    a.err = library_error_word();
    if (!a.err) return QK_ERR_CUDA;
    (void)max_len, (void)workspace_bytes;
    attn_rows_kernel<<<dim3(static_cast<unsigned>(B * max_q), n_q_heads), 128, 0,
                       reinterpret_cast<cudaStream_t>(stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? QK_OK : QK_ERR_CUDA;
}

}  // extern "C"
