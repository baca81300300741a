// qk_attn.cu -- attention over the 4-bit paged cache: the entry point, its
// argument checks, and how a call's rows and keys are cut over thread blocks.
// The kernels are in qk_attn_rows.cuh (few rows) and qk_attn_chunk.cu (many).
#include <atomic>
#include <cmath>

#include "qk_attn.cuh"
#include "qk_internal.h"

namespace qk {
using namespace attn;
namespace {

bool multiple(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool type_ok(int t) { return t == QK_F32 || t == QK_F16 || t == QK_BF16; }

// How a call's rows and keys are cut.
struct Cut {
    int pieces, sets, row_tile, tiles, splits;
    bool chunk;                      // the many-row form (qk_attn_chunk.cu)
    int64_t cut;                     // few rows: thread blocks that share all blocks (0: one a head)
    int64_t min_blocks, groups;      // groups: sequences * heads * tiles
};

std::atomic<int> g_skip_block{-1};

constexpr int64_t kChunkFrom = 64;           // rows a sequence and head from which it is taken
constexpr int64_t kCounters = 16384;         // ints at the start of every workspace, whatever the call
// max_len sizes the cut; no sequence is longer than `longest`.
Cut cut_for(int64_t B, int n_kv, int rep, int D, int64_t max_q, int64_t max_len, int64_t longest, bool fp32)
{
    Cut c{};
    const int64_t rows = max_q * rep;
    c.pieces = fp32 ? 2 : 1;
    c.chunk = !fp32 && rows >= kChunkFrom && D <= 128;
    // columns of a warp's tile: as few sets of 8 as hold the rows; with more sets a block of keys is taken apart once
    // for more rows (four sets of fp32 rows against one, 64 rows over 5000 keys: see the rule's measurements below)
    c.sets = 1;
    while (c.sets * 8 < rows * c.pieces && c.sets < (D <= 128 ? 4 : 2)) c.sets *= 2;
    c.row_tile = c.chunk ? kChunkRows : c.sets * 8 / c.pieces;
    c.tiles = static_cast<int>((rows + c.row_tile - 1) / c.row_tile);
    c.groups = B * n_kv * c.tiles;
    const int64_t blocks = (max_len + kBlockTokens - 1) / kBlockTokens;
    int sms = 152, smem = 0;
    device_limits(&sms, &smem);
    c.splits = 1;
    if (c.chunk) {
        // rounds of one thread block an SM, of key tiles of 8 blocks (about 1.2 us each) and 3 tiles' worth of start
        // and end; parts of several splits are written and read again (5 TB/s) by a second kernel (2 us)
        const int64_t tiles = (blocks + 7) / 8;
        double best = 1e30;
        for (int64_t rounds = 1, last = 0; rounds <= 8; ++rounds) {
            int64_t s = sms * rounds / c.groups;
            if (s * 2 > tiles) s = tiles / 2;
            if (s < 1) s = 1;
            if (s == last) continue;
            last = s;
            const double us = 1.2 * static_cast<double>((c.groups * s + sms - 1) / sms * ((tiles + s - 1) / s + 3)) +
                              (s > 1 ? 2.0 + 2e-7 * static_cast<double>(2 * s * c.groups * chunk_part_bytes(D)) : 0.0);
            if (us < best) best = us, c.splits = static_cast<int>(s);
        }
        c.min_blocks = (tiles + c.splits - 1) / c.splits * 8;
        if (c.min_blocks < 16) c.min_blocks = 16;
        return c;
    }
    // few rows: split where heads are at most half of the thread blocks that the GPU holds and have blocks to split,
    // over as many thread blocks as that.  (With more heads than that, one thread block a head: 512 heads of 8192
    // tokens take 146 us whole and 148, 160, 162 us in 2, 3, 4 parts.)
    const int64_t hold = static_cast<int64_t>(sms) * rows_blocks_per_sm(D / 32, c.sets);
    if (blocks > 2 * kWarps && c.groups * 2 <= hold && B * c.tiles <= kRowItems &&
        c.groups * ((longest + kBlockTokens - 1) / kBlockTokens) < (1 << 30))
        c.cut = hold;
    return c;
}

int64_t part_bytes_of(const Cut &c, int D)
{
    if (c.chunk) return chunk_part_bytes(D);
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
        max_len <= 0 || B > INT32_MAX / max_q)
        return 0;
    size_t most = 0;
    for (const bool fp32 : {true, false}) {
        const Cut c = cut_for(B, n_kv_heads, n_q_heads / n_kv_heads, head_dim, max_q, max_len, max_len, fp32);
        const size_t n = c.cut ? 4 * kCounters + c.cut * part_bytes_of(c, head_dim)
                               : c.splits > 1 ? 4 * kCounters + c.groups * c.splits * part_bytes_of(c, head_dim) : 0;
        if (n > most) most = n;
    }
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
    Cut cut = cut_for(B, n_kv, rep, D, max_q, max_len > 0 && max_len < keys ? max_len : keys, keys, q_type == QK_F32);
    // as many splits, or parts of thread blocks, as the workspace holds
    const int64_t room = workspace ? static_cast<int64_t>(workspace_bytes) - 4 * kCounters : 0;
    const int64_t fit = room > 0 ? room / part_bytes_of(cut, D) : 0;
    if (cut.splits > 1 && cut.splits > fit / cut.groups) cut.splits = fit / cut.groups > 1 ? static_cast<int>(fit / cut.groups) : 1;
    if (cut.cut > fit) cut.cut = fit > cut.groups ? fit : 0;
    const int64_t grid = cut.cut ? cut.cut : cut.groups * cut.splits;
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
    a.splits = cut.splits, a.min_blocks = static_cast<int>(cut.min_blocks < INT32_MAX ? cut.min_blocks : INT32_MAX);
    a.counters = static_cast<int *>(workspace);
    a.parts = reinterpret_cast<float *>(static_cast<char *>(workspace) + 4 * kCounters);
    a.err = library_error_word();
    a.wait_ns = library_wait_limit_ns();
    if (!a.err) return QK_ERR_CUDA;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaErrorInvalidValue;
    a.skip_block = g_skip_block.load();
    if (cut.chunk) return chunk_launch(a, D, cut.groups, s) == cudaSuccess ? QK_OK : QK_ERR_CUDA;
    switch (D) {
    case 64: e = rows_launch_64(a, cut.pieces, cut.sets, grid, s); break;
    case 96: e = rows_launch_96(a, cut.pieces, cut.sets, grid, s); break;
    case 128: e = rows_launch_128(a, cut.pieces, cut.sets, grid, s); break;
    case 256: e = rows_launch_256(a, cut.pieces, cut.sets, grid, s); break;
    }
    return e == cudaSuccess ? QK_OK : QK_ERR_CUDA;
}

}  // extern "C"
