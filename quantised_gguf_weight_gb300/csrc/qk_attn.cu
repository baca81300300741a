// qk_attn.cu -- attention over the 4-bit paged cache: the entry point, its
// argument checks, and how a call's rows and keys are cut over thread blocks.
// The kernels are in qk_attn_rows.cuh (few rows), qk_attn_chunk.cu and
// qk_attn_chunk32.cu (many).
#include <atomic>
#include <cmath>

#include "qk_attn_chunk.cuh"
#include "qk_internal.h"

namespace qk {
using namespace attn;
namespace {

bool multiple(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool type_ok(int t) { return t == QK_F32 || t == QK_F16 || t == QK_BF16; }

// How a call's rows and keys are cut.
struct Cut {
    int pieces, sets, row_tile, tiles, sms;
    bool chunk;                      // the many-row forms (qk_attn_chunk.cuh)
    int64_t cut;                     // thread blocks that share all blocks (0: one a head and row tile)
    int64_t groups;                  // sequences * heads * tiles
};

std::atomic<int> g_skip_block{-1};

// Rows a sequence and head from which it is taken.  Times of the few-row form and of it, us, heads of 128:
//   bf16, 8 sequences of 4096 tokens, 8 heads  16 rows 29 and 45, 32 41 and 45, 48 66 and 47, 256 248 and 68
//   bf16, 1 sequence of 16384, 8 heads         16 rows 21 and 27, 32 28 and 27, 48 38 and 28, 256 170 and 42
//   bf16, 8 of 4096, 32 heads of 96            16 rows 51 and 128, 32 96 and 128, 48 178 and 129
//   fp32, 8 of 4096, 8 heads                   16 rows 41 and 60, 32 54 and 61, 64 106 and 64, 128 209 and 69
constexpr int64_t kChunkFrom = 33;
constexpr int64_t kCounters = 16384;         // ints at the start of every workspace, whatever the call
constexpr int64_t kHead = 4 * kCounters + chunk::kPlanBytes;      // bytes before the parts
// max_len sizes the cut; no sequence is longer than `longest`.
Cut cut_for(int64_t B, int n_kv, int rep, int D, int64_t max_q, int64_t max_len, int64_t longest, int type)
{
    Cut c{};
    const bool fp32 = type == QK_F32;
    const int64_t rows = max_q * rep;
    int sms = 152, smem = 0;
    device_limits(&sms, &smem);
    c.sms = sms;
    c.pieces = fp32 ? 2 : 1;
    c.chunk = rows >= kChunkFrom && D <= 128;
    // Columns of a warp's tile, in sets of 8: a block of keys is taken apart once for all of them, but the more there
    // are the fewer thread blocks there are to fill the GPU.  fp32 rows have two columns each and take two sets at
    // once (16 columns, 16 short sequences: 15 us, one set 16), four where their heads and tiles still make three
    // quarters of the thread blocks that the GPU holds (8 x 32 rows over 4096 keys 54 us, two sets 58; 8 x 64 rows
    // over up to 5000 154 and 160).  16-bit rows take one, and two under the same condition: 64 x 16 rows over 4096
    // keys 122 us, one set 137; 64 x 32 rows 213, one 263, four 249; but 8 x 16 rows 32 us, one 29.
    c.sets = 1;
    for (int n = 2; n <= (fp32 && D <= 128 ? 4 : 2) && n * 4 < rows * c.pieces; n *= 2)
        if ((fp32 && n == 2) ||
            4 * B * n_kv * ((rows * c.pieces + n * 8 - 1) / (n * 8)) >= 3 * sms * rows_blocks_per_sm(D / 32, n))
            c.sets = n;
    c.row_tile = c.chunk ? (type == QK_BF16 ? kChunkRows : kChunkRows32) : c.sets * 8 / c.pieces;
    c.tiles = static_cast<int>((rows + c.row_tile - 1) / c.row_tile);
    c.groups = B * n_kv * c.tiles;
    const int64_t blocks = (max_len + kBlockTokens - 1) / kBlockTokens;
    if (c.chunk) {
        // one thread block an SM: heads are cut where they are few (and their items fit the cutting's tables), over at
        // most two for each.  Of one sequence the lengths are known here, and whether cutting it pays
        // (8 heads in 16 bits: 512 queries over 2048 keys whole 45 us, in two 51; 64 over 16384 whole 266 us, cut 42).
        const int64_t items = B * c.tiles;
        bool pays = items <= chunk::kItems && 2 * c.groups <= 3 * sms && 2 * sms <= chunk::kPlanBlocks &&
                    c.groups * ((longest + kBlockTokens - 1) / kBlockTokens) < (1 << 30);
        if (pays && B == 1) {
            const int most = static_cast<int>(blocks);
            const auto cost = [&](int k) {
                const int per = chunk::part_of(most, k);
                const int64_t parts = c.groups * ((most + per - 1) / per);
                return chunk::part_cost(static_cast<float>(c.groups * blocks), static_cast<int>(parts), per, sms,
                                        chunk_part_bytes(D, c.row_tile), k > 0);
            };
            bool better = false;
            for (int k = 1; k < chunk::kCutChoices; ++k) better |= cost(k) < cost(0);
            pays = better;
        }
        if (pays) c.cut = 2 * sms;
        return c;
    }
    // few rows: split where heads are at most a third of the thread blocks that the GPU holds and have blocks to split,
    // over as many thread blocks as that (304: 64 heads of 4096 tokens 27 us, whole 41; 128 heads 36 us, whole 29; 512
    // heads of 8192 whole 146, in 2, 3, 4 parts 148, 160, 162).
    const int64_t hold = static_cast<int64_t>(sms) * rows_blocks_per_sm(D / 32, c.sets);
    if (blocks > 2 * kWarps && c.groups * 3 <= hold && B * c.tiles <= kRowItems &&
        c.groups * ((longest + kBlockTokens - 1) / kBlockTokens) < (1 << 30))
        c.cut = hold;
    return c;
}

int64_t part_bytes_of(const Cut &c, int D)
{
    if (c.chunk) return chunk_part_bytes(D, c.row_tile);
    return (static_cast<int64_t>(c.row_tile) * D + 2 * c.row_tile) * 4;
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
        max_len < 0 || B > INT32_MAX / max_q)
        return 0;
    size_t most = 0;
    const auto of_length = [&](int64_t len) {
        for (const int type : {QK_F32, QK_F16, QK_BF16}) {
            const Cut c = cut_for(B, n_kv_heads, n_q_heads / n_kv_heads, head_dim, max_q, len, len, type);
            const size_t n = c.cut ? kHead + c.cut * part_bytes_of(c, head_dim) : 0;
            if (n > most) most = n;
        }
    };
    // a cut's bytes do not depend on the length, only whether there is one
    if (max_len > 0) of_length(max_len);
    else
        for (int64_t len = 256; len < INT32_MAX; len *= 2) of_length(len);
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
    Cut cut = cut_for(B, n_kv, rep, D, max_q, max_len > 0 && max_len < keys ? max_len : keys, keys, q_type);
    // as many parts as the workspace holds
    const int64_t room = workspace ? static_cast<int64_t>(workspace_bytes) - kHead : 0;
    const int64_t fit = room > 0 ? room / part_bytes_of(cut, D) : 0;
    if (cut.cut > fit) cut.cut = fit > cut.groups ? fit : 0;
    const int64_t grid = cut.cut ? cut.cut : cut.groups;
    if (grid > INT32_MAX) return QK_ERR_TOO_LARGE;
    AttnArgs a{};
    a.pages = static_cast<const uint8_t *>(cache->pages), a.n_pages = cache->n_pages;
    a.n_kv = n_kv, a.page_blocks = cache->page_tokens / kBlockTokens, a.rep = rep;
    a.q = q, a.ldq = ldq, a.q_type = q_type;
    a.page_table = page_table, a.ld_pages = ld_pages, a.max_pages = max_pages;
    a.lens = lens, a.q_start = q_start, a.T = T, a.max_q = max_q, a.window = window;
    a.scale_log2 = static_cast<float>(scale * 1.4426950408889634074);
    a.out = out, a.ldo = ldo, a.out_type = out_type;
    a.tiles = cut.tiles, a.items = static_cast<int>(B * cut.tiles), a.cut = static_cast<int>(cut.cut);
    a.sms = cut.sms;
    a.counters = static_cast<int *>(workspace);
    a.parts = reinterpret_cast<float *>(static_cast<char *>(workspace) + kHead);
    a.plan = static_cast<char *>(workspace) + 4 * kCounters;
    a.err = library_error_word();
    a.wait_ns = library_wait_limit_ns();
    if (!a.err) return QK_ERR_CUDA;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaErrorInvalidValue;
    a.skip_block = g_skip_block.load();
    if (cut.chunk) {
        e = q_type == QK_BF16 ? chunk_launch(a, D, cut.groups, s) : chunk32_launch(a, D, cut.groups, s);
        return e == cudaSuccess ? QK_OK : QK_ERR_CUDA;
    }
    switch (D) {
    case 64: e = rows_launch_64(a, cut.pieces, cut.sets, grid, s); break;
    case 96: e = rows_launch_96(a, cut.pieces, cut.sets, grid, s); break;
    case 128: e = rows_launch_128(a, cut.pieces, cut.sets, grid, s); break;
    case 256: e = rows_launch_256(a, cut.pieces, cut.sets, grid, s); break;
    }
    return e == cudaSuccess ? QK_OK : QK_ERR_CUDA;
}

}  // extern "C"
