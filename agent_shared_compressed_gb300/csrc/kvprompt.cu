// kvprompt.cu -- attention of whole prompts: every token of several sequences' new
// tokens over its own sequence's keys and values, causal, with a window and first
// tokens that stay visible, joined with attention over other tokens.
//
// For sequence b with n_b new tokens and T_b keys, new token i is at place
// p = T_b - n_b + i and sees t <= p, with a window w only t > p - w or t < z:
//   s_t = scale q . k_t,  out = sum_t softmax(s)_t v_t,  lse = log sum_t exp(s_t)
// joined: L = log(e^lse + e^base_lse), out = e^(lse-L) out + e^(base_lse-L) base.
#include <algorithm>
#include <cmath>

#include "kvp_internal.cuh"

namespace kvp {

// Weights are relative to 2^PT_BIAS times the largest, so that sums of values up to bf16's
// largest stay finite.
constexpr float PT_BIAS = 40.0f;

struct PromptArgs {
    const uint16_t *q, *k, *v;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;  // strides in elements
    const int32_t *q_first, *k_first, *k_lens;
    const float *base_out, *base_lse;
    uint16_t *out;
    float *lse;
    uint32_t *error;
    float scale2;  // scale * log2(e)
    int nseq, n, nk, nq, H, G, window, sinks;
};

__device__ __forceinline__ void prompt_flag(const PromptArgs &a, uint32_t f) {
    if (a.error) atomicOr(a.error, f);
}

// A sequence's new tokens and keys; n = 0 where its numbers lie outside the tensors.
struct PromptSeq {
    int first, n, k_first, T;
};
__device__ __forceinline__ PromptSeq prompt_seq(const PromptArgs &a, int b, bool flag) {
    PromptSeq s;
    s.first = int(ld_plain_u32(a.q_first + b));
    const int end = int(ld_plain_u32(a.q_first + b + 1));
    s.k_first = int(ld_plain_u32(a.k_first + b)), s.T = int(ld_plain_u32(a.k_lens + b));
    s.n = end - s.first;
    if (s.first < 0 || end < s.first || end > a.n || s.k_first < 0 || s.T < 0 || int64_t(s.k_first) + s.T > a.nk) {
        if (flag) prompt_flag(a, FLAG_PAGE);
        s.n = 0;
    }
    return s;
}

// What a row ends with: the weights of its own result (already divided by its sum)
// and of the base, and its lse.
__device__ __forceinline__ float2 prompt_join(const PromptArgs &a, uint64_t row, float lse, bool writes) {
    float wa = 1.0f, wb = 0.0f;
    if (a.base_lse) {
        const float bl = a.base_lse[row];
        if (!(lse == -INFINITY && bl == -INFINITY)) {
            const float top = fmaxf(lse, bl);
            const float ea = expf(lse - top), eb = expf(bl - top), tot = ea + eb;
            wa = ea / tot, wb = eb / tot;
            lse = top + logf(tot);
        }
    }
    if (writes && a.lse) a.lse[row] = lse;
    return make_float2(wa, wb);
}

// One row by one warp, a key at a time in fp32: lane l holds dims l d/32 ...  The keys are
// those of [k0, k1) that the row at place p sees.  acc is relative to 2^ref.
template <int D>
__device__ __forceinline__ void row_keys(const PromptArgs &a, const float (&q)[D / 32], const uint16_t *k, const uint16_t *v,
                                         int p, int64_t k0, int64_t k1, float (&acc)[D / 32], float &ref, float &sum) {
    constexpr int VPL = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t old = a.window ? int64_t(p) - a.window + 1 : 0;  // the oldest token of the window
    for (int64_t t = k0; t < min(k1, int64_t(p) + 1); ++t) {
        if (t < old && t >= a.sinks) {
            t = min(old, k1) - 1;
            continue;
        }
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) s = fmaf(q[i], __uint_as_float(uint32_t(k[t * a.k_ts + lane * VPL + i]) << 16), s);
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        s *= a.scale2;
        const float top = fmaxf(ref, s), f = ref == -INFINITY ? 0.0f : exp2f(ref - top);
        const float w = exp2f(s - (top == -INFINITY ? 0.0f : top) - PT_BIAS);
        ref = top, sum = fmaf(sum, f, w);
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            acc[i] = fmaf(acc[i], f, w * __uint_as_float(uint32_t(v[t * a.v_ts + lane * VPL + i]) << 16));
    }
}

template <int D>
__global__ void __launch_bounds__(128) prompt_rows(const __grid_constant__ PromptArgs a) {
    constexpr int VPL = D / 32;
    const int lane = threadIdx.x & 31;
    const uint32_t w = blockIdx.x * 4u + (threadIdx.x >> 5);
    if (w >= uint32_t(a.n) * uint32_t(a.nq)) return;
    const int tok = int(w / uint32_t(a.nq)), j = int(w % uint32_t(a.nq)), h = j / a.G;
    for (int b = 0; b < a.nseq; ++b) {
        const PromptSeq s = prompt_seq(a, b, lane == 0);
        if (tok < s.first || tok >= s.first + s.n) continue;
        float q[VPL], acc[VPL], ref = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            q[i] = __uint_as_float(uint32_t(a.q[tok * a.q_ts + j * a.q_hs + lane * VPL + i]) << 16);
            acc[i] = 0.0f;
        }
        row_keys<D>(a, q, a.k + s.k_first * a.k_ts + h * a.k_hs, a.v + s.k_first * a.v_ts + h * a.v_hs, s.T - s.n + tok - s.first,
                    0, s.T, acc, ref, sum);
        const uint64_t row = uint64_t(tok) * uint32_t(a.nq) + uint32_t(j);
        const float2 f = prompt_join(a, row, sum > 0.0f ? (ref + PT_BIAS + log2f(sum)) * 0.69314718055994531f : (sum == 0.0f ? -INFINITY : sum), lane == 0);
        const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            float y = acc[i] * inv * f.x;
            if (a.base_out && f.y != 0.0f) y = fmaf(f.y, a.base_out[row * D + lane * VPL + i], y);
            reinterpret_cast<__nv_bfloat16 *>(a.out)[row * D + lane * VPL + i] = __float2bfloat16_rn(y);
        }
        return;
    }
}

static int prompt_ok(const kvp_prompt_shape *s) {
    if (!s) return KVP_ERR_ARG;
    if (s->n_seqs < 0 || s->n_q_tokens < 0 || s->n_k_tokens < 0 || s->n_q_heads <= 0 || s->n_kv_heads <= 0 ||
        s->n_q_heads % s->n_kv_heads != 0)
        return KVP_ERR_ARG;
    if (s->head_dim != 64 && s->head_dim != 128) return KVP_ERR_UNSUPPORTED_D;
    if (s->n_seqs > KVP_PROMPT_MAX_SEQS || s->n_q_heads > 65536 || s->n_q_heads / s->n_kv_heads > 128) return KVP_ERR_SIZE;
    if (int64_t(s->n_q_tokens) * s->n_q_heads >= (int64_t(1) << 31)) return KVP_ERR_SIZE;
    return KVP_OK;
}

static int rows_ok(const kvp_rows *r, int tokens, int heads) {
    if (!r || (!r->ptr && tokens > 0)) return KVP_ERR_ARG;
    if (!aligned(r->ptr, 16) || r->token_stride % 8 != 0 || r->head_stride % 8 != 0) return KVP_ERR_ALIGN;
    constexpr int64_t MOST = int64_t(1) << 38;  // elements: a copy's stride is below 2^40 bytes
    if ((tokens > 1 && (r->token_stride <= 0 || r->token_stride >= MOST)) ||
        (heads > 1 && (r->head_stride <= 0 || r->head_stride >= MOST)))
        return KVP_ERR_ARG;
    return KVP_OK;
}

}  // namespace kvp

using namespace kvp;

extern "C" {

size_t kvprompt_workspace_bytes(const kvp_prompt_shape *shape) {
    if (prompt_ok(shape) != KVP_OK) return 0;
    return 256;
}

int kvprompt_attend(const kvp_prompt_shape *shape, const kvp_rows *q, const kvp_rows *k, const kvp_rows *v,
                    const int32_t *q_first, const int32_t *k_first, const int32_t *k_lens, float scale, int window,
                    int sinks, const float *base_out, const float *base_lse, void *out, float *lse, uint32_t *error,
                    void *ws, size_t ws_bytes, void *stream) {
    int rc = prompt_ok(shape);
    if (rc != KVP_OK) return rc;
    if (window < 0 || sinks < 0 || !std::isfinite(scale)) return KVP_ERR_ARG;
    if (!q_first || !k_first || !k_lens || !out || !ws || (base_out == nullptr) != (base_lse == nullptr)) return KVP_ERR_ARG;
    if ((rc = rows_ok(q, shape->n_q_tokens, shape->n_q_heads)) != KVP_OK) return rc;
    if ((rc = rows_ok(k, shape->n_k_tokens, shape->n_kv_heads)) != KVP_OK) return rc;
    if ((rc = rows_ok(v, shape->n_k_tokens, shape->n_kv_heads)) != KVP_OK) return rc;
    if (!aligned(q_first, 4) || !aligned(k_first, 4) || !aligned(k_lens, 4) || !aligned(base_out, 16) ||
        !aligned(base_lse, 4) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(error, 4) || !aligned(ws, 16))
        return KVP_ERR_ALIGN;
    if (ws_bytes < kvprompt_workspace_bytes(shape)) return KVP_ERR_SIZE;
    if (shape->n_seqs == 0 || shape->n_q_tokens == 0) return KVP_OK;
    PromptArgs a;
    a.q = static_cast<const uint16_t *>(q->ptr), a.q_ts = q->token_stride, a.q_hs = q->head_stride;
    a.k = static_cast<const uint16_t *>(k->ptr), a.k_ts = k->token_stride, a.k_hs = k->head_stride;
    a.v = static_cast<const uint16_t *>(v->ptr), a.v_ts = v->token_stride, a.v_hs = v->head_stride;
    a.q_first = q_first, a.k_first = k_first, a.k_lens = k_lens;
    a.base_out = base_out, a.base_lse = base_lse;
    a.out = static_cast<uint16_t *>(out), a.lse = lse, a.error = error;
    a.scale2 = scale * 1.4426950408889634f;
    a.nseq = shape->n_seqs, a.n = shape->n_q_tokens, a.nk = shape->n_k_tokens;
    a.nq = shape->n_q_heads, a.H = shape->n_kv_heads, a.G = a.nq / a.H;
    a.window = window, a.sinks = sinks;
    const unsigned rows = unsigned(a.n) * unsigned(a.nq);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (shape->head_dim == 128)
        prompt_rows<128><<<(rows + 3) / 4, 128, 0, st>>>(a);
    else
        prompt_rows<64><<<(rows + 3) / 4, 128, 0, st>>>(a);
    count_launch();
    return launch_status();
}

int kvprompt_status(const uint32_t *error, void *stream) {
    if (!error) return KVP_ERR_ARG;
    if (!aligned(error, 4)) return KVP_ERR_ALIGN;
    uint32_t f = 0;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cudaMemcpyAsync(&f, error, sizeof f, cudaMemcpyDeviceToHost, st) != cudaSuccess) return KVP_ERR_CUDA;
    if (cudaStreamSynchronize(st) != cudaSuccess) return KVP_ERR_CUDA;
    return flags_to_status(f);
}

}  // extern "C"
