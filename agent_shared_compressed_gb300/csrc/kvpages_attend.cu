// kvpages_attend.cu -- attention over pages: the entry points, and the kernels
// without a window (kvpages_attend.cuh) for all formats but 4-bit keys.
#include "kvpages_attend.cuh"

namespace kvp {

static thread_local uint32_t g_next_polls = 0, g_next_lanes = 0;
static thread_local bool g_limit_next = false;

template int launch_attend<128, KVP_PAGES_BF16, false>(PagesAttendArgs &, int, cudaStream_t);
template int launch_attend<64, KVP_PAGES_BF16, false>(PagesAttendArgs &, int, cudaStream_t);
template int launch_attend<128, KVP_PAGES_K8V8, false>(PagesAttendArgs &, int, cudaStream_t);
template int launch_attend<64, KVP_PAGES_K8V8, false>(PagesAttendArgs &, int, cudaStream_t);
template int launch_attend<128, KVP_PAGES_K8V4, false>(PagesAttendArgs &, int, cudaStream_t);
template int launch_attend<64, KVP_PAGES_K8V4, false>(PagesAttendArgs &, int, cudaStream_t);

// compiled in kvpages_attend_4bit.cu and kvpages_attend_window.cu
extern template int launch_attend<128, KVP_PAGES_K4V4, false>(PagesAttendArgs &, int, cudaStream_t);
extern template int launch_attend<64, KVP_PAGES_K4V4, false>(PagesAttendArgs &, int, cudaStream_t);
extern template int launch_attend<128, KVP_PAGES_BF16, true>(PagesAttendArgs &, int, cudaStream_t);
extern template int launch_attend<64, KVP_PAGES_BF16, true>(PagesAttendArgs &, int, cudaStream_t);
extern template int launch_attend<128, KVP_PAGES_K8V8, true>(PagesAttendArgs &, int, cudaStream_t);
extern template int launch_attend<64, KVP_PAGES_K8V8, true>(PagesAttendArgs &, int, cudaStream_t);
extern template int launch_attend<128, KVP_PAGES_K8V4, true>(PagesAttendArgs &, int, cudaStream_t);
extern template int launch_attend<64, KVP_PAGES_K8V4, true>(PagesAttendArgs &, int, cudaStream_t);
extern template int launch_attend<128, KVP_PAGES_K4V4, true>(PagesAttendArgs &, int, cudaStream_t);
extern template int launch_attend<64, KVP_PAGES_K4V4, true>(PagesAttendArgs &, int, cudaStream_t);

template <int FMT>
static int launch_format(PagesAttendArgs &a, int rows, bool d128, bool win, cudaStream_t st) {
    if (win) return d128 ? launch_attend<128, FMT, true>(a, rows, st) : launch_attend<64, FMT, true>(a, rows, st);
    return d128 ? launch_attend<128, FMT, false>(a, rows, st) : launch_attend<64, FMT, false>(a, rows, st);
}

static int attend_counts_ok(const kvp_pages_config *cfg, int n_seqs, int n_q_tokens, int n_q_heads) {
    const int rc = pages_ok(cfg);
    if (rc != KVP_OK) return rc;
    if (n_seqs < 0 || n_q_tokens <= 0 || n_q_heads <= 0 || n_q_heads % cfg->n_kv_heads != 0) return KVP_ERR_ARG;
    if (n_seqs > KVP_PAGES_MAX_SEQS || n_q_tokens > 64 || n_q_heads > 65536) return KVP_ERR_SIZE;
    if (int64_t(n_seqs) * n_q_tokens * n_q_heads >= (int64_t(1) << 31)) return KVP_ERR_SIZE;
    return KVP_OK;
}

// Workspace: the plan, the partial rows' statistics, the partial rows.
struct AttendWs {
    uint64_t stats, part, total;
};
static AttendWs attend_ws(const kvp_pages_config *cfg, int n_seqs, int n_q_tokens, int n_q_heads) {
    const uint64_t rows =
        uint64_t(attend_grid()) * PAT_MOST_WARPS * 2u * uint64_t(tile_rows(n_q_tokens * (n_q_heads / cfg->n_kv_heads), cfg->format));
    AttendWs w;
    w.stats = align256(4ull * uint64_t(n_seqs + 1));
    w.part = w.stats + align256(rows * 8ull);
    w.total = w.part + rows * uint64_t(cfg->head_dim) * 4ull;
    return w;
}

}  // namespace kvp

using namespace kvp;

extern "C" {

size_t kvpages_attend_workspace_bytes(const kvp_pages_config *cfg, int n_seqs, int n_q_tokens, int n_q_heads) {
    if (attend_counts_ok(cfg, n_seqs, n_q_tokens, n_q_heads) != KVP_OK) return 0;
    return size_t(attend_ws(cfg, n_seqs, n_q_tokens, n_q_heads).total);
}

int kvp_test_limit_next_pages_attend_lanes(uint32_t polls, uint32_t lanes) {
    g_next_polls = polls, g_next_lanes = lanes;
    g_limit_next = true;
    return KVP_OK;
}

int kvp_test_limit_next_pages_attend(uint32_t polls) {
    return kvp_test_limit_next_pages_attend_lanes(polls, 0xFFFFFFFFu);
}

int kvpages_attend(const void *pages, const kvp_pages_config *cfg, int layer, int n_seqs, int n_q_tokens,
                   int n_q_heads, const void *q, float scale, const int32_t *table, int max_pages,
                   const int32_t *lens, const float *base_out, const float *base_lse, void *out, float *lse, void *ws,
                   size_t ws_bytes, void *stream) {
    return kvpages_attend_window(pages, cfg, layer, n_seqs, n_q_tokens, n_q_heads, q, scale, 0, 0, table, max_pages, lens,
                                 base_out, base_lse, out, lse, ws, ws_bytes, stream);
}

int kvpages_attend_window(const void *pages, const kvp_pages_config *cfg, int layer, int n_seqs, int n_q_tokens,
                          int n_q_heads, const void *q, float scale, int window, int sinks, const int32_t *table,
                          int max_pages, const int32_t *lens, const float *base_out, const float *base_lse, void *out,
                          float *lse, void *ws, size_t ws_bytes, void *stream) {
    const int rc = attend_counts_ok(cfg, n_seqs, n_q_tokens, n_q_heads);
    if (rc != KVP_OK) return rc;
    if (!pages || layer < 0 || layer >= cfg->n_layers || max_pages <= 0 || window < 0 || sinks < 0) return KVP_ERR_ARG;
    if (!q || !table || !lens || !out || !ws || (base_out == nullptr) != (base_lse == nullptr)) return KVP_ERR_ARG;
    if (!std::isfinite(scale)) return KVP_ERR_ARG;
    if (!aligned(pages, 256) || !aligned(q, 16) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(base_out, 16) ||
        !aligned(base_lse, 4) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(ws, 16))
        return KVP_ERR_ALIGN;
    const AttendWs w = attend_ws(cfg, n_seqs, n_q_tokens, n_q_heads);
    if (ws_bytes < w.total) return KVP_ERR_SIZE;
    // unit counts are 32-bit
    const unsigned __int128 blocks = (unsigned __int128)uint32_t(max_pages) * uint32_t(cfg->page_tokens / 16) * uint32_t(n_seqs);
    if (blocks >> 31) return KVP_ERR_SIZE;
    if (n_seqs == 0) return KVP_OK;
    PagesAttendArgs a;
    a.pv = pages_view(const_cast<void *>(pages), *cfg, layer);
    a.q = static_cast<const uint16_t *>(q);
    a.table = table, a.lens = lens, a.base_out = base_out, a.base_lse = base_lse;
    a.out = static_cast<uint16_t *>(out), a.lse = lse;
    a.plan = static_cast<uint32_t *>(ws);
    a.stats = reinterpret_cast<float2 *>(static_cast<uint8_t *>(ws) + w.stats);
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + w.part);
    a.scale2 = scale * 1.4426950408889634f;
    a.nseq = n_seqs, a.m = n_q_tokens, a.nq = n_q_heads, a.G = n_q_heads / cfg->n_kv_heads;
    a.R = n_q_tokens * a.G;
    const int rows = tile_rows(a.R, cfg->format);
    a.RT = (a.R + rows - 1) / rows;
    a.max_pages = max_pages;
    a.window = window, a.sinks = sinks;
    a.polls = g_limit_next ? g_next_polls : PAT_WAIT_LIMIT;
    a.poll_lanes = g_limit_next ? g_next_lanes : 0xFFFFFFFFu;
    g_limit_next = false;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool d128 = cfg->head_dim == 128, win = window > 0;
    switch (cfg->format) {
        case KVP_PAGES_BF16: return launch_format<KVP_PAGES_BF16>(a, rows, d128, win, st);
        case KVP_PAGES_K8V8: return launch_format<KVP_PAGES_K8V8>(a, rows, d128, win, st);
        case KVP_PAGES_K8V4: return launch_format<KVP_PAGES_K8V4>(a, rows, d128, win, st);
        default: return launch_format<KVP_PAGES_K4V4>(a, rows, d128, win, st);
    }
}

}  // extern "C"
