// kvpages_attend.cu -- attention of each sequence's newest tokens over its
// pages, joined with attention over other tokens (the shared pool's).
//
// For sequence b, query token i, query head j (KV head h = j / (nq / H)):
//   s_t = scale q . k_t,  t < len_b - (m - 1 - i)
//   out = sum_t softmax(s)_t v_t,  lse = log sum_t exp(s_t)
// joined: L = log(e^lse + e^base_lse), out = e^(lse-L) out + e^(base_lse-L) base.
//
// One block per (sequence, query token, query head): a lane quad takes every
// 32nd token with its own running maximum and sum, and the block's quads are
// merged at the end.
#include <cmath>

#include "kvp_pages.cuh"

namespace kvp {

constexpr int PAT_THREADS = 128;

struct PagesAttendArgs {
    PagesView pv;
    const uint16_t *q;
    const int32_t *table, *lens;
    const float *base_out, *base_lse;
    uint16_t *out;
    float *lse;
    float scale2;  // scale * log2(e)
    int m, nq, max_pages;
};

template <int D, int FMT>
__global__ void __launch_bounds__(PAT_THREADS) pages_attend(const __grid_constant__ PagesAttendArgs a) {
    using B = Block<D, FMT>;
    constexpr int NB = D / 32, NQD = PAT_THREADS / 4;
    __shared__ float st[NQD][2];
    __shared__ float acc_s[NQD][D + 1];
    const int quad = threadIdx.x >> 2, tig = threadIdx.x & 3;
    const uint64_t row = blockIdx.x;  // (b, i, j)
    const int j = int(row % uint32_t(a.nq)), i = int(row / uint32_t(a.nq) % uint32_t(a.m));
    const uint32_t b = uint32_t(row / (uint64_t(a.nq) * uint32_t(a.m)));
    const int h = j / (a.nq / a.pv.H);
    if (!pages_match(a.pv)) {
        if (threadIdx.x == 0) pages_flag(a.pv, FLAG_HEADER);
        return;
    }
    int len = max(a.lens[b], 0);
    if (int64_t(len) > int64_t(a.max_pages) << a.pv.logP) {
        if (threadIdx.x == 0) pages_flag(a.pv, FLAG_PAGE);
        len = int(int64_t(a.max_pages) << a.pv.logP);
    }
    len = max(0, len - (a.m - 1 - i));
    float q[NB][8], acc[NB][8];
#pragma unroll
    for (int g = 0; g < NB; ++g) {
        const uint4 v = *reinterpret_cast<const uint4 *>(a.q + row * D + 32 * g + 8 * tig);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) q[g][2 * k] = bf16_lo(w[k]), q[g][2 * k + 1] = bf16_hi(w[k]);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[g][k] = 0.0f;
    }
    float mx = -INFINITY, l = 0.0f;
    for (int t = quad; t < (len + NQD - 1) / NQD * NQD; t += NQD) {
        const uint8_t *src = nullptr;
        if (t < len) {
            const int page = a.table[uint64_t(b) * uint32_t(a.max_pages) + uint32_t(t >> a.pv.logP)];
            if (page >= 0 && page < a.pv.n_pages)
                src = a.pv.layer + uint64_t(page) * a.pv.page_bytes + uint64_t(h) * a.pv.tile_bytes +
                      uint64_t((uint32_t(t) & uint32_t(a.pv.P - 1)) / PAGES_BLOCK) * B::BYTES;
            else if (tig == 0)
                pages_flag(a.pv, FLAG_PAGE);
        }
        float x[NB][8], s = 0.0f;
        if (src) {
            load_key_row<D, FMT>(src, uint32_t(t) % PAGES_BLOCK, tig, x);
#pragma unroll
            for (int g = 0; g < NB; ++g)
#pragma unroll
                for (int k = 0; k < 8; ++k) s = fmaf(q[g][k], x[g][k], s);
        }
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        if (!src) continue;
        s *= a.scale2;
        const float m2 = fmaxf(mx, s), ref = m2 == -INFINITY ? 0.0f : m2;
        const float f = exp2f(mx - ref), p = exp2f(s - ref);
        mx = m2;
        l = l * f + p;
        load_value_row<D, FMT>(src, uint32_t(t) % PAGES_BLOCK, tig, x);
#pragma unroll
        for (int g = 0; g < NB; ++g)
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[g][k] = acc[g][k] * f + p * x[g][k];
    }
    if (tig == 0) st[quad][0] = mx, st[quad][1] = l;
#pragma unroll
    for (int g = 0; g < NB; ++g)
#pragma unroll
        for (int k = 0; k < 8; ++k) acc_s[quad][32 * g + 8 * tig + k] = acc[g][k];
    __syncthreads();
    float M = -INFINITY, L = 0.0f, o = 0.0f;
    for (int k = 0; k < NQD; ++k) M = fmaxf(M, st[k][0]);
    const float ref = M == -INFINITY ? 0.0f : M;
    if (threadIdx.x < D) {
        for (int k = 0; k < NQD; ++k) {
            const float f = exp2f(st[k][0] - ref);
            L += f * st[k][1];
            o += f * acc_s[k][threadIdx.x];
        }
        o = L > 0.0f ? o / L : 0.0f;
        float lse = L > 0.0f ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
        if (a.base_out) {
            const float bl = a.base_lse[row], top = fmaxf(lse, bl);
            if (top > -INFINITY) {
                const float wa = expf(lse - top), wb = expf(bl - top);
                o = (wa * o + wb * a.base_out[row * D + threadIdx.x]) / (wa + wb);
                lse = top + logf(wa + wb);
            }
        }
        reinterpret_cast<__nv_bfloat16 *>(a.out)[row * D + threadIdx.x] = __float2bfloat16_rn(o);
        if (threadIdx.x == 0 && a.lse) a.lse[row] = lse;
    }
}

template <int D, int FMT>
static int launch_attend(const PagesAttendArgs &a, unsigned grid, cudaStream_t st) {
    pages_attend<D, FMT><<<grid, PAT_THREADS, 0, st>>>(a);
    count_launch();
    return launch_status();
}

static int attend_counts_ok(const kvp_pages_config *cfg, int n_seqs, int n_q_tokens, int n_q_heads) {
    const int rc = pages_ok(cfg);
    if (rc != KVP_OK) return rc;
    if (n_seqs < 0 || n_q_tokens <= 0 || n_q_heads <= 0 || n_q_heads % cfg->n_kv_heads != 0) return KVP_ERR_ARG;
    if (n_seqs > 8192 || n_q_tokens > 64 || n_q_heads > 65536) return KVP_ERR_SIZE;
    if (int64_t(n_seqs) * n_q_tokens * n_q_heads >= (int64_t(1) << 31)) return KVP_ERR_SIZE;
    return KVP_OK;
}

}  // namespace kvp

using namespace kvp;

extern "C" {

size_t kvpages_attend_workspace_bytes(const kvp_pages_config *cfg, int n_seqs, int n_q_tokens, int n_q_heads) {
    if (attend_counts_ok(cfg, n_seqs, n_q_tokens, n_q_heads) != KVP_OK) return 0;
    return 256;
}

int kvpages_attend(const void *pages, const kvp_pages_config *cfg, int layer, int n_seqs, int n_q_tokens,
                   int n_q_heads, const void *q, float scale, const int32_t *table, int max_pages,
                   const int32_t *lens, const float *base_out, const float *base_lse, void *out, float *lse, void *ws,
                   size_t ws_bytes, void *stream) {
    const int rc = attend_counts_ok(cfg, n_seqs, n_q_tokens, n_q_heads);
    if (rc != KVP_OK) return rc;
    if (!pages || layer < 0 || layer >= cfg->n_layers || max_pages <= 0) return KVP_ERR_ARG;
    if (!q || !table || !lens || !out || !ws || (base_out == nullptr) != (base_lse == nullptr)) return KVP_ERR_ARG;
    if (!std::isfinite(scale)) return KVP_ERR_ARG;
    if (!aligned(pages, 256) || !aligned(q, 16) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(base_out, 16) ||
        !aligned(base_lse, 4) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(ws, 16))
        return KVP_ERR_ALIGN;
    if (ws_bytes < kvpages_attend_workspace_bytes(cfg, n_seqs, n_q_tokens, n_q_heads)) return KVP_ERR_SIZE;
    if (n_seqs == 0) return KVP_OK;
    PagesAttendArgs a;
    a.pv = pages_view(const_cast<void *>(pages), *cfg, layer);
    a.q = static_cast<const uint16_t *>(q);
    a.table = table, a.lens = lens, a.base_out = base_out, a.base_lse = base_lse;
    a.out = static_cast<uint16_t *>(out), a.lse = lse;
    a.scale2 = scale * 1.4426950408889634f;
    a.m = n_q_tokens, a.nq = n_q_heads, a.max_pages = max_pages;
    const unsigned grid = unsigned(n_seqs) * unsigned(n_q_tokens) * unsigned(n_q_heads);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool d128 = cfg->head_dim == 128;
    switch (cfg->format) {
        case KVP_PAGES_BF16:
            return d128 ? launch_attend<128, KVP_PAGES_BF16>(a, grid, st) : launch_attend<64, KVP_PAGES_BF16>(a, grid, st);
        case KVP_PAGES_K8V8:
            return d128 ? launch_attend<128, KVP_PAGES_K8V8>(a, grid, st) : launch_attend<64, KVP_PAGES_K8V8>(a, grid, st);
        default:
            return d128 ? launch_attend<128, KVP_PAGES_K8V4>(a, grid, st) : launch_attend<64, KVP_PAGES_K8V4>(a, grid, st);
    }
}

}  // extern "C"
